"""What the memory model asks of the ragged products' source, where no run can show that it is missing (no GPU needed)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "mxfp8_block_scaled_routed_b200", "csrc")


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _code(text):
    return re.sub(r"//[^\n]*", "", text)


def test_cleared_rows_are_released_to_the_other_cta():
    """The weight gradient's tail rows are written by one CTA of a pair and read by products that a thread of the other CTA
    issues: the arrival that announces them releases at cluster scope, behind a proxy fence of every lane, and the issuer
    acquires at cluster scope."""
    ragged, sm100 = _code(_read("ragged.cuh")), _code(_read("sm100.cuh"))
    clear = ragged[ragged.index("warp == 3) {\n    \n    if constexpr (kMode == kWgrad)"):ragged.index("else if (warp >= 4)")]
    assert re.search(r"fence_proxy_async\(\);\s*__syncwarp\(\);\s*if \(lane == 0\) mbar_arrive_release_shared\(full_bar\(stage\), 0\);", clear)
    helper = sm100[sm100.index("void mbar_arrive_release_shared"):]
    assert re.search(r"fence\.release\.sync_restrict::shared::cta\.cluster;.*mbarrier\.arrive\.relaxed\.cluster\.shared::cluster", helper[:helper.index("\n}")], re.S)
    assert "mbar_wait_cluster(full_bar(stage), phase)" in ragged
    wait = sm100[sm100.index("bool mbar_try_wait_cluster"):]
    assert "try_wait.parity.acquire.cluster" in wait[:wait.index("\n}")]
