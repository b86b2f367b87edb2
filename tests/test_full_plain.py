"""The plain 64-bit forms that the full-attention tests compare with: against
torch's own attention and against finite differences (no GPU needed)."""
import torch

import full_plain as fp


def _inputs(Lq, Lk, Hq, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return r(Lq, Hq, d), r(Lk, Hkv, d), r(Lk, Hkv, d), r(Lq, Hq, d)


def test_plain_prefill_equals_masked_attention():
    for Lq, Lk, Hq, Hkv in ((7, 7, 4, 2), (3, 9, 6, 2), (1, 5, 2, 2)):
        q, k, v, _ = _inputs(Lq, Lk, Hq, Hkv, 16, Lq)
        out = fp.prefill(q, [k], [v], [(0, Lq)], 0.25, torch.float32)[0]
        seen = torch.arange(Lk)[None] <= torch.arange(Lq)[:, None] + (Lk - Lq)
        kk, vv = (x.repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=seen, scale=0.25)
        assert torch.allclose(out, want.transpose(0, 1), atol=1e-12)


def test_plain_rows_without_keys():
    q, k, v, _ = _inputs(5, 3, 2, 1, 8, 1)
    out, lse = fp.prefill(q, [k], [v], [(0, 5)], 0.3, torch.float32)[:2]
    assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all() and lse[2:].isfinite().all()
    out, lse = fp.prefill(q, [k[:0]], [v[:0]], [(0, 5)], 0.3, torch.float32)[:2]
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_plain_backward_equals_differences():
    q, k, v, dout = _inputs(6, 9, 4, 2, 8, 2)
    scale = 0.4
    fwd = lambda q, k, v: fp.prefill(q, [k], [v], [(0, 6)], scale, torch.float32)  # noqa: E731
    out, lse = fwd(q, k, v)[:2]
    grads, _ = fp.backward(q, k, v, out, dout, lse, scale, torch.float32)
    g = torch.Generator().manual_seed(3)
    for n, x in enumerate((q, k, v)):
        u = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        at = lambda t: [y + t * u if m == n else y for m, y in enumerate((q, k, v))]  # noqa: E731
        diff = ((fwd(*at(h))[0] - fwd(*at(-h))[0]) * dout).sum() / (2 * h)
        assert abs(diff - (grads[n] * u).sum()) <= 1e-7 * (1 + abs(diff))
