"""The bench's DRAM traffic figure belongs to the sources that it names: when
one of them changes, the figure is taken again (the bench reports null until then)."""


def test_the_traffic_figure_is_of_the_present_sources():
    import bench
    assert bench.STA_FWD_TRAFFIC_SRC_SHA == bench._src_sha()
