"""The tracked profiles of the headline kernel were measured on the sources that are here: the
benchmark reports them only for sources of the same hash."""

import json

import pytest

import bench


@pytest.mark.parametrize("path, field", [(bench.TRAFFIC_FILE, "hbm_bytes_per_launch_mean"),
                                         (bench.TRACE_FILE, "trace_us_per_launch_mean")])
def test_profiles_belong_to_the_sources(path, field):
    profile = json.load(open(path))
    assert profile["kernel_source_hash"] == bench.kernel_source_hash()
    assert profile[field] > 0
