"""The attention traffic that bench.py reports was captured on the sources that
are there: once they change, take the two captures again (the commands are in
profiles/k_attend_llama8b_128k.md) or drop the figure."""
import bench


def test_the_traffic_figure_belongs_to_the_current_sources():
    assert bench.ATTEND_TRAFFIC["sources_sha256"] == bench.attend_sources_digest()
