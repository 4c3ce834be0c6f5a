"""The ABI version counts the entry points around the cache (major * 100 + minor)."""

import paged_kv_cache_144_gb300 as pa


def test_version_is_that_of_the_operators_around_the_cache():
    assert pa.pa_version() == 101
