"""Waits of the tcgen05 kernels.  What they order, and what becomes of a launch one of
whose waits runs out, cannot be seen from results, so their source is read; the
pairs of CTAs of the 8-bit floating point path are then run again and again
beside each other."""
import os
import re

import pytest
import torch

from projection_gemm_gb300 import build, skg
from tests import f8_reference as R


def kernel_source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    return src[src.index("__global__"):]


def test_waits_of_a_pair_are_at_cluster_scope():
    """Both CTAs of a pair arrive at full, empty, afull and aempty, so a pair waits there with cluster scope."""
    src = kernel_source("skg_f8_wide.cu")
    assert not re.findall(r"mbar_wait\(&(full|empty|afull|aempty)\b", src)
    assert set(re.findall(r"\bwait\(&(\w+)\[", src)) == {"full", "empty", "afull", "aempty"}
    pair, single = re.search(r"auto wait = .*?if constexpr \(PAIR == 2\)\s*return (\w+)\(.*?else\s*return (\w+)\(", src, re.S).groups()
    assert (pair, single) == ("mbar_wait_cluster", "mbar_wait")


@pytest.mark.parametrize("name,fail,landed,before", [
    ("skg_f8_split.cu", "f8_fail", "mbar_wait(&full[", "tmem_dealloc"),
    ("skg_f8_wide.cu", "f8_fail", "wait_landed()", "cluster_sync();"),
    ("skg_q8_split.cu", "q8_fail", "mbar_wait(&wfull[", "tmem_dealloc"),
    ("skg_q8_wide.cu", "q8_fail", "wait_landed()", "cluster_sync();"),
    ("skg_splitk_tc.cu", "record_failure", "mbar_wait(&full[", "tmem_dealloc"),
    ("skg_group_tc.cu", "group_failure", "wait_landed()", "tmem_dealloc")])
def test_copies_land_before_a_cta_that_aborts_leaves(name, fail, landed, before):
    """Whoever raises the abort flag may do so long after the producer's last copy, so the flag is looked at when every
    role has ended; and before exit, or, where a peer's copies are counted here, before the pair's last barrier."""
    src = kernel_source(name)
    src = src[:src.index("\ncudaError_t ")]
    met = src.index("__syncthreads();", src.rindex(fail + "("))
    looked = re.search(r"if \([^{;]*flags\[0\]\)", src[met:])
    assert looked
    looked = met + looked.start()
    assert looked < src.index(landed, looked) < src.index(before, met)
    assert not re.search(r"if \([^{;&]*flags\[0\]\) \{", src[:met])      # and not only sooner


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,split,E", [(5000, 2100, 512, 1, 0), (700, 1032, 4112, 3, 0), (3000, 520, 1040, 1, 7),
                                           (256, 256, 4096, 4, 0)])
def test_pairs_give_the_same_bits_while_others_run(M, N, K, split, E):
    """Two streams of pairs, each accumulator used many times over: every run has the bits of the first, which is right."""
    build.build()
    g = torch.Generator().manual_seed(M + K)
    each = (E,) if E else ()
    x, W = ((torch.randn(*s, generator=g) * 100).clamp(-448, 448).to(R.F8).cuda() for s in ((M, K), (*each, N, K)))
    xs = torch.rand(M, R.blocks(K), generator=g).cuda()
    ws = torch.rand(*each, R.blocks(N), R.blocks(K), generator=g).cuda()
    offsets = None
    if E:
        cuts = torch.sort(torch.randint(0, M + 1, (E - 1,), generator=g)).values.tolist()
        offsets = torch.tensor([0, *cuts, M], dtype=torch.int32, device="cuda")
    plan = skg.F8Plan(M, N, K, "bf16", experts=E)
    plan.force(skg.SKG_F8_KERNEL_WIDE, 256, split)
    want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    plan.run(x, xs, W, ws, None, want, offsets=offsets)
    plan.check()
    bounds = offsets.tolist() if E else [0, M]
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            R.check_linear(x[a:b], xs[a:b], W[e] if E else W, ws[e] if E else ws, None, want[a:b])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ys = [[torch.zeros_like(want) for _ in range(12)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(12):
        for s, y in zip(streams, ys):
            plan.run(x, xs, W, ws, None, y[i], offsets=offsets, stream=s)
    torch.cuda.synchronize()
    plan.check()
    assert all(torch.equal(t, want) for y in ys for t in y)
