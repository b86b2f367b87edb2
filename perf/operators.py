"""The paged cache and full-attention operators as work to be measured: real
calls over their range, each in a plain form (elementary torch operations in
32 bits) and as the calls a user makes of the library.

    append    msa_paged_append: rotate q and k by position, write k and v to pages
    decode    msa_full_attn_decode: one query token per sequence over a paged cache
    prefill   msa_full_attn_prefill: causal attention over packed sequences
    chunk     msa_full_attn_prefill_paged: new tokens of prompts over a paged prefix
    backward  msa_full_attn_backward: dq, dk, dv of prefill
"""
import math
import random

import torch

own = False  # True: run() calls the library; False: the plain form

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# (query heads, key/value heads, head dim): the library's own workload shapes, and other ratios it is built for
HEADS = [(32, 8, 128), (8, 2, 64), (16, 2, 64), (4, 4, 64), (6, 2, 128), (16, 1, 128), (8, 8, 128)]


def listed():
    h128 = {"Hq": 32, "Hkv": 8, "d": 128}
    return [
        # one step of a serving loop: the new token of each of 64 sequences joins its cache (latency)
        {"name": "append_step", "op": "append", "dtype": "bf16", "B": 64, "lo": 1, "hi": 1, "old_lo": 0,
         "old_hi": 4000, "page": 64, "rot": 128, "interleaved": False, "mix": 1, **h128},
        # a batch of ragged prompts enters its cache, some behind a prefix that is there already
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "B": 12, "lo": 1, "hi": 4096, "old_lo": 0,
         "old_hi": 1000, "page": 64, "rot": 128, "interleaved": False, "mix": 2, **h128},
        # the smallest decode: one user, a short context (latency)
        {"name": "decode_one", "op": "decode", "dtype": "bf16", "B": 1, "lo": 777, "hi": 777, "page": 16, "mix": 3,
         **h128},
        # a serving batch with contexts from 4K to 128K: the cache's whole length is read
        {"name": "decode_b16_128k", "op": "decode", "dtype": "bf16", "B": 16, "lo": 4096, "hi": 131072, "page": 64,
         "mix": 4, **h128},
        # fp32 decode, small heads, odd lengths from one token on
        {"name": "decode_fp32", "op": "decode", "dtype": "fp32", "B": 9, "lo": 1, "hi": 5001, "page": 32, "mix": 5,
         "Hq": 8, "Hkv": 2, "d": 64},
        # many short prompts packed together: tiles that end inside sequences
        {"name": "prefill_short", "op": "prefill", "dtype": "bf16", "B": 24, "lo": 1, "hi": 700, "mix": 6, "Hq": 16,
         "Hkv": 2, "d": 64},
        # one whole prompt of 8K tokens
        {"name": "prefill_8k", "op": "prefill", "dtype": "bf16", "B": 1, "lo": 8192, "hi": 8192, "mix": 7, **h128},
        # chunked prompts: some hundred new tokens each behind 8K to 16K tokens in the cache
        {"name": "chunk_paged", "op": "chunk", "dtype": "bf16", "B": 4, "lo": 200, "hi": 1024, "old_lo": 8000,
         "old_hi": 16000, "page": 64, "mix": 8, **h128},
        # fp32 prompts of odd lengths
        {"name": "prefill_fp32", "op": "prefill", "dtype": "fp32", "B": 3, "lo": 100, "hi": 999, "mix": 9, "Hq": 8,
         "Hkv": 2, "d": 64},
        # training on short documents packed into one row
        {"name": "backward_short", "op": "backward", "dtype": "bf16", "B": 10, "lo": 1, "hi": 900, "mix": 10,
         "Hq": 8, "Hkv": 2, "d": 64},
        # training on one document of 8K tokens
        {"name": "backward_8k", "op": "backward", "dtype": "bf16", "B": 1, "lo": 8192, "hi": 8192, "mix": 11, **h128},
        # fp32 gradients of odd lengths
        {"name": "backward_fp32", "op": "backward", "dtype": "fp32", "B": 3, "lo": 50, "hi": 500, "mix": 12, "Hq": 8,
         "Hkv": 2, "d": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill", "chunk", "backward"])
    Hq, Hkv, d = rng.choice(HEADS)
    c = {"op": op, "dtype": "fp32" if rng.random() < 0.2 else "bf16", "Hq": Hq, "Hkv": Hkv, "d": d,
         "mix": rng.randrange(1 << 20)}
    small = c["dtype"] == "fp32"
    if op == "append":
        c["hi"] = 1 if rng.random() < 0.3 else _log(rng, 1, 4096)
        c["B"] = _log(rng, 1, 256 if c["hi"] == 1 else max(1, min(64, 30000 // c["hi"])))
        c["lo"] = rng.choice([1, c["hi"]])
        c["old_lo"], c["old_hi"] = 0, _log(rng, 1, 3000)
        c["rot"] = rng.choice([16, d // 2, d])
        c["interleaved"] = rng.random() < 0.4
    elif op == "decode":
        c["hi"] = _log(rng, 1, 4000 if small else 131072)
        c["B"] = _log(rng, 1, max(1, min(128, int(8e9) // (c["hi"] * Hkv * d * 8))))
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
    else:
        # scores of the padded batch: at most those of the largest listed prompt
        most = 8192 * 8192 * 32 // (256 if small else 2)
        c["hi"] = _log(rng, 1, 700 if small else 6000)
        if op == "chunk":
            c["hi"] = min(c["hi"], 1500)
            c["old_lo"], c["old_hi"] = 0, _log(rng, 1, 1500 if small else 12000)
        each = Hq * c["hi"] * (c["hi"] + c.get("old_hi", 0))
        while each > most:
            c["hi"] = c["hi"] * 2 // 3
            each = Hq * c["hi"] * (c["hi"] + c.get("old_hi", 0))
        c["B"] = _log(rng, 1, max(1, min(48, most // each)))
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
    if op in ("append", "decode", "chunk"):
        c["page"] = rng.choice([16, 32, 64, 128])
    return c


def _lengths(case):
    """(tokens per sequence the call brings, tokens its cache holds before them)."""
    r = random.Random(case["mix"])
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    old = [r.randint(case.get("old_lo", 0), case.get("old_hi", 0)) for _ in range(case["B"])]
    return new, old


def _pairs(n, old):
    """Visible (query, key) pairs of n tokens behind `old` earlier ones."""
    return n * old + n * (n + 1) // 2


def work(case):
    new, old = _lengths(case)
    Hq, Hkv, d, e = case["Hq"], case["Hkv"], case["d"], 2 if case["dtype"] == "bf16" else 4
    T, keys = sum(new), sum(new) + sum(old)
    pairs = sum(_pairs(n, o) for n, o in zip(new, old))
    op = case["op"]
    if op == "append":
        rows = max(n + o for n, o in zip(new, old)) - min(old)
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * d * e + min(rows, T) * case["rot"] * 4,
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    if op == "decode":
        return {"bytes": T * 2 * Hkv * d * e + case["B"] * Hq * (2 * d * e + 4), "flops": 4 * T * Hq * d}
    if op in ("prefill", "chunk"):
        return {"bytes": keys * 2 * Hkv * d * e + T * Hq * (2 * d * e + 4), "flops": 4 * pairs * Hq * d}
    return {"bytes": keys * 4 * Hkv * d * e + T * Hq * (4 * d * e + 4), "flops": 10 * pairs * Hq * d}


def prepare(case, seed):
    """A user's tensors before the call: packed tokens with their offsets, or
    the cache's pages with the table that says which sequence holds which."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    new, old = _lengths(case)
    B, Hq, Hkv, d, op = case["B"], case["Hq"], case["Hkv"], case["d"], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32 if dt == torch.float32 else dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def offsets(v):
        at = [0]
        for n in v:
            at.append(at[-1] + n)
        return ints(at)

    s = {"case": case, "new": new, "old": old, "cu": offsets(new), "T": sum(new), "longest": max(new)}
    if op in ("append", "decode", "chunk"):
        ps = case["page"]
        # the cache: a sequence's pages lie anywhere in it; entries past its last page are -1
        total = [n + o for n, o in zip(new, old)]
        need = [-(-n // ps) for n in total]
        num_pages = sum(need) + 3
        order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32).tolist()
        table, at = [], 0
        for n in need:
            table.append(order[at:at + n] + [-1] * (max(need) - n))
            at += n
        s["table"] = ints(table)
        s["kv_len"] = ints(total)
        s["k_cache"], s["v_cache"] = normal(num_pages, ps, Hkv, d), normal(num_pages, ps, Hkv, d)
        s["keys"] = max(total)
    if op == "append":
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["q"], s["k"], s["v"] = normal(s["T"], Hq, d), normal(s["T"], Hkv, d), normal(s["T"], Hkv, d)
    elif op == "decode":
        s["q"] = normal(B, Hq, d)
    else:
        s["q"] = normal(s["T"], Hq, d)
        if op != "chunk":
            s["k"], s["v"] = normal(s["T"], Hkv, d), normal(s["T"], Hkv, d)
            s["keys"] = s["longest"]
        if op == "backward":  # a training step has the forward's output and lse in hand, and the output's gradient
            s["dout"] = normal(s["T"], Hq, d)
            s["out"], s["lse"] = _plain_prefill(s)
    return s


# ---- the plain forms ---------------------------------------------------------
def _where(cu, T):
    """(sequence, index within it) of every packed token."""
    t = torch.arange(T, dtype=torch.int64, device=cu.device)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return b, t - cu[b]


def _plain_append(s):
    case = s["case"]
    half, ps = case["rot"] // 2, case["page"]
    b, i = _where(s["cu"], s["T"])
    n_new = s["cu"][1:] - s["cu"][:-1]
    pos = (s["kv_len"] - n_new)[b].long() + i
    c, sn = s["rope"][pos][:, None, :, 0], s["rope"][pos][:, None, :, 1]

    def rotate(x):
        y = x.float()
        if case["interleaved"]:
            a, z = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            r = torch.stack([a * c - z * sn, z * c + a * sn], -1).flatten(-2)
        else:
            a, z = y[..., :half], y[..., half:2 * half]
            r = torch.cat([a * c - z * sn, z * c + a * sn], -1)
        return torch.cat([r, y[..., 2 * half:]], -1).to(x.dtype)

    slot = s["table"][b, pos // ps].long() * ps + pos % ps
    s["k_cache"].flatten(0, 1)[slot] = rotate(s["k"])
    s["v_cache"].flatten(0, 1)[slot] = s["v"]
    return rotate(s["q"]), s["k_cache"], s["v_cache"]


def _plain_attend(q, k, v, visible, scale):
    """q [B, Lq, Hq, d], k and v [B, Lk, Hkv, d] (fp32), visible [B, Lq, Lk] -> out, lse [B, Lq, Hq]."""
    B, Lq, Hq, d = q.shape
    Hkv = k.shape[2]
    qg = q.reshape(B, Lq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, hpg * Lq, d]
    sc = torch.matmul(qg, k.permute(0, 2, 3, 1)) * scale
    sc = sc.view(B, Hkv, Hq // Hkv, Lq, -1).masked_fill_(~visible[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True).clamp_min_(-1e30)
    p = sc.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).view(B, Hkv, Hq // Hkv, Lq, d) / den.clamp_min(1e-30)
    lse = (m + den.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, d), lse.permute(0, 3, 1, 2).reshape(B, Lq, Hq)


def _pages(s):
    """The padded batch's keys and values [B, keys, Hkv, d] out of the pages."""
    at = s["table"].clamp_min(0).long()
    return tuple(s[x][at].flatten(1, 2)[:, :s["keys"]].float() for x in ("k_cache", "v_cache"))


def _plain_decode(s):
    k, v = _pages(s)
    j = torch.arange(s["keys"], device=k.device)
    seen = j[None, None] < s["kv_len"][:, None, None]
    o, lse = _plain_attend(s["q"].float()[:, None], k, v, seen, s["case"]["d"] ** -0.5)
    return o[:, 0].to(s["q"].dtype), lse[:, 0]


def _plain_prefill(s):
    """Packed rows spread to a padded batch, attention there, rows back."""
    q, cu = s["q"], s["cu"]
    b, i = _where(cu, s["T"])
    n = (cu[1:] - cu[:-1]).long()
    rows = (cu[:-1, None].long() + torch.arange(s["longest"], device=q.device)).clamp_max_(s["T"] - 1)
    if "table" in s:
        (k, v), total = _pages(s), s["kv_len"].long()
    else:
        k, v, total = s["k"][rows].float(), s["v"][rows].float(), n
    pos = (total - n)[:, None] + torch.arange(s["longest"], device=q.device)
    j = torch.arange(s["keys"], device=q.device)
    seen = (j[None, None] <= pos[:, :, None]) & (j[None, None] < total[:, None, None])
    o, lse = _plain_attend(q[rows].float(), k, v, seen, s["case"]["d"] ** -0.5)
    return o[b, i].to(q.dtype), lse[b, i].contiguous()


def _plain_backward(s):
    q, cu, scale = s["q"], s["cu"], s["case"]["d"] ** -0.5
    Hkv, d = s["case"]["Hkv"], s["case"]["d"]
    hpg = s["case"]["Hq"] // Hkv
    b, i = _where(cu, s["T"])
    n = (cu[1:] - cu[:-1]).long()
    t = torch.arange(s["longest"], device=q.device)
    rows = (cu[:-1, None].long() + t).clamp_max_(s["T"] - 1)
    B, L = rows.shape
    seen = (t[None, None] <= t[None, :, None]) & (t[None, :, None] < n[:, None, None])

    def grouped(x):  # [T, Hq, d] -> [B, Hkv, hpg * L, d]
        return x[rows].float().view(B, L, Hkv, hpg, d).permute(0, 2, 3, 1, 4).flatten(2, 3)

    delta = (s["out"].float() * s["dout"].float()).sum(-1)
    per_row = [x[rows].view(B, L, Hkv, hpg).permute(0, 2, 3, 1).flatten(2, 3)[..., None] for x in (s["lse"], delta)]
    qg, dog = grouped(q), grouped(s["dout"])
    k, v = (s[x][rows].float().permute(0, 2, 1, 3) for x in ("k", "v"))
    p = torch.matmul(qg, k.transpose(-1, -2)).mul_(scale).sub_(per_row[0]).exp_()
    p.view(B, Hkv, hpg, L, L).masked_fill_(~seen[:, None, None], 0.0)
    dv = torch.matmul(p.transpose(-1, -2), dog)
    ds = torch.matmul(dog, v.transpose(-1, -2)).sub_(per_row[1]).mul_(p)
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(-1, -2), qg).mul_(scale)
    dq = dq.view(B, Hkv, hpg, L, d).permute(0, 3, 1, 2, 4).reshape(B, L, Hkv * hpg, d)
    return dq[b, i].to(q.dtype), dk.permute(0, 2, 1, 3)[b, i].to(q.dtype), dv.permute(0, 2, 1, 3)[b, i].to(q.dtype)


# ---- the library's calls -----------------------------------------------------
def _scratch(s, op, Nq, Nk):
    """The workspace a user's program allocates once for its sizes."""
    import block_sparse_long_select_gb300 as msa

    if "ws" not in s:
        c = s["case"]
        code = msa.MSA_BF16 if c["dtype"] == "bf16" else msa.MSA_FP32
        s["ws"] = msa.workspace(msa.msa_workspace_size(getattr(msa, op), c["B"], Nq, Nk, c["Hkv"], c["Hq"], c["d"], 0,
                                                       0, 0, code), s["q"].device)
    return s["ws"]


def _own_append(s):
    import block_sparse_long_select_gb300 as msa

    ws = _scratch(s, "MSA_OP_PAGED_APPEND", s["T"], 0)
    one = s["case"]["lo"] == s["case"]["hi"] == 1  # one token per sequence: no offsets needed
    q = msa.msa_paged_append(s["q"], s["k"], s["v"], s["rope"], None if one else s["cu"], s["kv_len"], s["table"],
                             s["k_cache"], s["v_cache"], interleaved=s["case"]["interleaved"], ws=ws)
    return q, s["k_cache"], s["v_cache"]


def _own_decode(s):
    import block_sparse_long_select_gb300 as msa

    ws = _scratch(s, "MSA_OP_FULL_DECODE", 1, s["table"].shape[1] * s["case"]["page"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    return msa.msa_full_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"], lse=lse, ws=ws), lse


def _own_prefill(s):
    import block_sparse_long_select_gb300 as msa

    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    if "table" in s:
        ws = _scratch(s, "MSA_OP_FULL_PREFILL", s["T"], s["table"].shape[1] * s["case"]["page"])
        return msa.msa_full_attn_prefill_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                                               lse=lse, ws=ws), lse
    ws = _scratch(s, "MSA_OP_FULL_PREFILL", s["T"], s["T"])
    return msa.msa_full_attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["cu"], lse=lse, ws=ws), lse


def _own_backward(s):
    import block_sparse_long_select_gb300 as msa

    ws = _scratch(s, "MSA_OP_FULL_BACKWARD", s["T"], s["T"])
    return msa.msa_full_attn_backward(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["cu"], s["cu"], ws=ws)


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "prefill": _own_prefill, "chunk": _own_prefill,
                "backward": _own_backward}[op](s)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill, "chunk": _plain_prefill,
            "backward": _plain_backward}[op](s)


# ---- the definition in 64 bits, sequence by sequence and head by head -----------
def exact(case, seed):
    s = prepare(case, seed)
    new, old = s["new"], s["old"]
    Hq, Hkv, d, op = case["Hq"], case["Hkv"], case["d"], case["op"]
    hpg, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    starts = [sum(new[:b]) for b in range(case["B"])]
    dev = s["q"].device
    if op == "append":
        ps, half = case["page"], case["rot"] // 2
        out = s["q"].double()
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for b, (t0, n, o) in enumerate(zip(starts, new, old)):
            cs = torch.complex(*(s["rope"][o:o + n, :, x].double() for x in (0, 1)))[:, None]
            turned = []
            for x in (s["q"][t0:t0 + n].double(), s["k"][t0:t0 + n].double()):
                y = x.clone()
                if case["interleaved"]:
                    z = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * cs
                    y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * cs
                    y[..., :half], y[..., half:2 * half] = z.real, z.imag
                turned.append(y)
            out[t0:t0 + n] = turned[0]
            table = s["table"][b].tolist()
            for p in range(o // ps, (o + n - 1) // ps + 1):  # page by page
                lo, hi = max(o, p * ps), min(o + n, (p + 1) * ps)
                kc[table[p], lo - p * ps:hi - p * ps] = turned[1][lo - o:hi - o]
                vc[table[p], lo - p * ps:hi - p * ps] = s["v"][t0 + lo - o:t0 + hi - o].double()
        return out, kc, vc
    if op == "decode":
        starts, new, old = list(range(case["B"])), [1] * case["B"], [n - 1 for n in new]
    T = s["q"].shape[0]
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(T, Hq, dtype=torch.float64, device=dev)
    grads = [torch.zeros(T, h, d, dtype=torch.float64, device=dev) for h in (Hq, Hkv, Hkv)]
    for b, (t0, n, o) in enumerate(zip(starts, new, old)):
        mine = slice(t0, t0 + n)
        late = torch.ones(n, n + o, dtype=torch.bool, device=dev).triu(o + 1) if n > 1 else None
        if "table" in s:
            used = s["table"][b, :-(-(n + o) // case["page"])].long()
        for g in range(Hkv):
            if "table" in s:
                k, v = (s[x][used, :, g].reshape(-1, d)[:n + o].double() for x in ("k_cache", "v_cache"))
            else:
                k, v = s["k"][mine, g].double(), s["v"][mine, g].double()
            for h in range(g * hpg, (g + 1) * hpg):
                q = s["q"][mine, h].double()
                x = (q @ k.T) * scale
                if late is not None:
                    x[late] = -math.inf
                if op != "backward":
                    lse[mine, h] = torch.logsumexp(x, 1)
                    out[mine, h] = torch.softmax(x, 1) @ v
                    continue
                do = s["dout"][mine, h].double()
                p = torch.exp(x - s["lse"][mine, h].double()[:, None])
                ds = p * (do @ v.T - (do * s["out"][mine, h].double()).sum(1)[:, None])
                grads[0][mine, h] = scale * (ds @ k)
                grads[1][mine, g] += scale * (ds.T @ q)
                grads[2][mine, g] += p.T @ do
    return tuple(grads) if op == "backward" else (out, lse)
