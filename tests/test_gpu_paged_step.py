"""avsg_rotary_write in front of the sparse step: its k and v rows go to the
host store with avsg_append, its fp32 queries to avsg_step, without a copy or
a change of layout between them; the step then follows the oracle on the same
rows (one and three tokens per step)."""
import numpy as np
import pytest
import torch

import paged_reference as ref
import workload as W
from gpu_harness import ATTN_TOL, Parity

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,tokens", [("batch", 1), ("mtp", 3)])
def test_rotary_then_append_and_step(name, tokens):
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    steps, live0 = 4, 4000
    w = W.get_workload(name, steps=steps, requests=3, kv_heads=2, context=4096, k=200, slots=1024)
    assert w.tokens_per_step == tokens
    sel = W.selections(w.replace(context=live0), steps)
    p = Parity(w, steps=steps, sel=sel, initial_entries=live0)
    R, H, G, D = w.requests, w.kv_heads, w.q_per_kv, w.head_dim
    T = R * tokens
    freq = rotary_frequencies(D)
    gen = torch.Generator("cuda").manual_seed(5)
    rows = PagedCache.allocate(1, 1, T, H, 1, D)          # k and v, a row per token
    new = [torch.empty(R * H, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    try:
        for t in range(steps):
            qkv = torch.randn(T, (H * G + 2 * H) * D, generator=gen, device="cuda").to(torch.bfloat16)
            q, k, v = qkv.split((H * G * D, H * D, H * D), 1)
            pos = torch.tensor([live0 + t + j for _ in range(R) for j in range(tokens)],
                               dtype=torch.int32, device="cuda")
            q_out = torch.empty(R * H, tokens, G, D, dtype=torch.float32, device="cuda")
            rows.rotary(q, k, v, pos, None, freq.cuda(), q_out, tokens_per_request=tokens)
            assert rows.error()[0] == 0
            # the first token of each request joins the store: [requests][kv-heads][D]
            for x, y in zip((rows.k, rows.v), new):
                y.copy_(x[0, ::tokens, :, 0].reshape(R * H, D))
            p.sess.append(*new)
            p.ref.append(*(x.view(torch.int16).cpu().numpy().view(np.uint16) for x in new))
            p.sel[t][:, :, 0] = live0 + t                  # every token selects it
            p.q[t] = q_out.cpu().numpy()
            p.step(t)
            # and the queries are the definition's
            x = q.double().cpu().numpy().reshape(T, H * G, D)
            want = ref.rotate(x, ref.turns_of(pos.tolist(), freq.numpy().view(np.uint64)), D, 0, False, 1.0)
            want = want.reshape(R, tokens, H, G, D).transpose(0, 2, 1, 3, 4).reshape(R * H, tokens, G, D)
            assert np.abs(p.q[t] - want).max() <= 6e-7 * 2 * np.abs(x).max() + 2.0**-24 * np.abs(want).max()
        assert p.sess.stats().device_error == 0 and p.max_err <= ATTN_TOL
    finally:
        p.close()
