"""The routed-experts profile pages were taken on the kernel sources as they are."""
import os
import re

import pytest

import bench

PAGES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "profiles")


@pytest.mark.parametrize("page", ["routed_experts.md", "routed_experts_tiles.md"])
def test_the_page_names_the_sources_it_was_taken_on(page):
    text = open(os.path.join(PAGES, page), encoding="utf-8").read()
    line = next(l for l in text.splitlines() if l.startswith("Sources: "))
    files = re.findall(r"`(fl_\w+\.\w+)`", line)
    assert {"fl_grouped.hpp", "fl_grouped_dma.hpp", "fl_grouped_inst.hip", "fl_moe.hip", "fl_moe.hpp"} <= set(files)
    assert re.search(r"`([0-9a-f]{16})`", line).group(1) == bench.source_hash(files), f"{page} is stale: profile again"
