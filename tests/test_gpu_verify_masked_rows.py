"""verify_mss and verify_naive on target rows whose masked tokens hold very low finite logits, in runs longer than the range of
the vocabulary that a warp walks: the oracle's tokens."""
import numpy as np
import pytest
import torch

import oracle
from tree_speculative_verification_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [-1e30, -3.4028234e38, -1e6])
@pytest.mark.parametrize("T", [1.0, 0.5])
def test_masked_ranges(masked, T):
    B, n, V = 16, 4, 4096
    rng = np.random.default_rng(11)
    logits = rng.normal(0, 3, (B, n, V)).astype(np.float32)
    for b in range(B):
        lo = int(rng.integers(0, V - 300))
        keep = np.zeros(V, bool)
        keep[lo:lo + 300] = rng.random(300) < 0.5
        keep[lo] = True
        logits[b, :, ~keep] = masked
    x = logits.astype(np.float64) + rng.normal(0, 1, logits.shape)
    ssm = np.where(logits == np.float32(masked), 0.0, np.exp(np.clip(x - x.max(-1, keepdims=True), -100, 0)))
    ssm = (ssm / ssm.sum(-1, keepdims=True)).astype(np.float32)
    parent = np.tile(np.arange(-1, n - 1, dtype=np.int32), (B, 1))
    tokens = np.zeros((B, n), np.int32)
    for b in range(B):
        for v in range(1, n):
            tokens[b, v] = rng.choice(np.flatnonzero(ssm[b, v - 1]))
    nodes, uni = np.full(B, n, np.int32), rng.random((B, 2, n), dtype=np.float32)
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    t = api.Tree(B, n)
    api.tree_build(t, cu(tokens), cu(parent), cu(nodes))
    for naive in (False, True):
        out, path, count, low = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((B, n + 1), (B, n + 1), (B,), (B,)))
        if naive:
            api.verify_naive(out, path, count, cu(logits), cu(uni), T, t, lowmargin=low)
            ref = oracle.verify_naive(logits, parent, tokens, nodes, uni, T)
        else:
            api.verify_mss(out, path, count, cu(logits), cu(ssm), cu(parent), cu(uni), T, t, lowmargin=low)
            ref = oracle.verify_mss(logits, ssm, parent, uni, parent, tokens, nodes, T)
        assert int((low > 0).sum()) <= 2
        for b in range(B):
            c = int(ref["count"][b])
            if not low[b]:
                assert int(count[b]) == c and out[b, :c].tolist() == ref["tokens"][b, :c].tolist(), (naive, b)
