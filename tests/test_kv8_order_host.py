"""How the tile kernel over 8-bit caches hands rank 1's halves of K, V and Q to rank 0, which issues the products of both
CTAs: read from the source, since a missing order between two CTAs need not show in any run."""
import os
import re

from video_diffusion_transformer_rope_gb300 import _build


def _source():
    return re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, "attn_tiles_sm103.cu")).read())


def test_no_arrival_of_cta_scope_announces_plain_stores_to_the_other_cta():
    text = _source()
    assert "mbar_arrive_remote_release" not in text and "release.cta.shared::cluster" not in text
    # the converters' part: they arrive in their own CTA alone
    part = text[text.index("regs_decrease<kRegsConvert>"):text.index("regs_decrease<k8 ? kRegsCtl8 : kRegsCtl>")]
    assert "mapa_shared" not in part and "mbar_arrive_remote" not in part
    assert len(re.findall(r"fence_proxy_async_smem\(\);\s*(?:\}\s*)?__syncwarp\(\);\s*if \(lane == 0\)", part)) == 3


def test_rank_0_acquires_at_cluster_scope_what_the_converters_wrote():
    text = _source()
    issuer = text[text.index("constexpr uint32_t kIdQK"):text.index("mma_commit_pair_warp(sCtl + kBarDone)")]
    assert "warp_wait<k8>(bar" in issuer
    waits = re.findall(r"(\w+)\((?:sCtl \+ kBar[KV]Full|q_full)", issuer)
    assert len(waits) == 5 and set(waits) == {"wait_tile"}
    relay = text[text.index("mma_commit_pair_warp(sCtl + kBarDone)"):text.index("tma_prefetch_desc(&tm_q)")]
    assert re.search(r"if \(k8\)\s*mbar_arrive_remote_cluster\(mapa_shared\(bar, 0\)\);\s*else\s*mbar_arrive_remote\(", relay)
