"""Caches in 8 bits and shared prefixes as work to be measured: real calls over
their range, each in a plain form (elementary torch operations in 32 bits) and
as the calls a user makes of the library.

    append   msa_paged_append_fp8: rotate q and k by position, write k and v to pages
             as e4m3 with a scale per (token, head); then msa_paged_read_fp8 of the
             new tokens, which says what the pages stand for
    read     msa_paged_read_fp8: cached keys and values as packed rows
    decode   msa_full_attn_decode_fp8: one query token per sequence over such a cache
    shared   msa_full_attn_decode_shared: the same over bf16 / fp32 pages, for groups
             of sequences that begin with the same pages

An e4m3 row stands for code * scale; scale is the smallest power of two, at
least 2^-126, with max|row| / scale <= 448 (0 for a row of zeros).
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
        # fp32 tokens, part of the head rotated, pairs side by side, odd lengths
        {"name": "append_fp32", "op": "append", "dtype": "fp32", "B": 7, "lo": 1, "hi": 901, "old_lo": 0,
         "old_hi": 300, "page": 16, "rot": 32, "interleaved": True, "mix": 3, "Hq": 8, "Hkv": 2, "d": 64},
        # the prefixes of four chunked prompts come back as rows for a prefill
        {"name": "read_prefixes", "op": "read", "dtype": "bf16", "B": 4, "lo": 8000, "hi": 16000, "page": 64, "mix": 4,
         **h128},
        # short odd caches as fp32 rows (latency)
        {"name": "read_short_fp32", "op": "read", "dtype": "fp32", "B": 37, "lo": 1, "hi": 120, "page": 32, "mix": 5,
         "Hq": 8, "Hkv": 2, "d": 64},
        # the smallest decode: one user, a short context (latency)
        {"name": "decode_one", "op": "decode", "dtype": "bf16", "B": 1, "lo": 777, "hi": 777, "page": 16, "mix": 6,
         **h128},
        # a serving batch with contexts from 4K to 128K: the cache's whole length is read
        {"name": "decode_b16_128k", "op": "decode", "dtype": "bf16", "B": 16, "lo": 4096, "hi": 131072, "page": 64,
         "mix": 7, **h128},
        # fp32 queries, small heads, odd lengths from one token on
        {"name": "decode_fp32", "op": "decode", "dtype": "fp32", "B": 9, "lo": 1, "hi": 5001, "page": 32, "mix": 8,
         "Hq": 8, "Hkv": 2, "d": 64},
        # 32 samples of one prompt of 8K tokens, some tokens on
        {"name": "shared_samples", "op": "shared", "dtype": "bf16", "B": 32, "P": 1, "pre_lo": 8192, "pre_hi": 8192,
         "lo": 1, "hi": 200, "alone": 0, "page": 64, "mix": 9, **h128},
        # 96 conversations behind three system prompts, and one without any
        {"name": "shared_prompts", "op": "shared", "dtype": "bf16", "B": 97, "P": 3, "pre_lo": 1000, "pre_hi": 8192,
         "lo": 50, "hi": 2500, "alone": 1, "page": 16, "mix": 10, **h128},
        # questions about one long document
        {"name": "shared_128k", "op": "shared", "dtype": "bf16", "B": 24, "P": 1, "pre_lo": 131072, "pre_hi": 131072,
         "lo": 1, "hi": 1000, "alone": 0, "page": 128, "mix": 11, **h128},
        # fp32, small heads, short
        {"name": "shared_fp32", "op": "shared", "dtype": "fp32", "B": 10, "P": 2, "pre_lo": 64, "pre_hi": 600, "lo": 1,
         "hi": 300, "alone": 2, "page": 16, "mix": 12, "Hq": 8, "Hkv": 2, "d": 64},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "shared"])
    Hq, Hkv, d = rng.choice(HEADS)
    c = {"op": op, "dtype": "fp32" if rng.random() < 0.2 else "bf16", "Hq": Hq, "Hkv": Hkv, "d": d,
         "page": rng.choice([16, 32, 64, 128]), "mix": rng.randrange(1 << 20)}
    small = c["dtype"] == "fp32"
    if op == "append":
        c["hi"] = 1 if rng.random() < 0.3 else _log(rng, 1, 4096)
        c["B"] = _log(rng, 1, 256 if c["hi"] == 1 else max(1, min(64, 30000 // c["hi"])))
        c["old_lo"], c["old_hi"] = 0, _log(rng, 1, 3000)
        c["rot"] = rng.choice([16, d // 2, d])
        c["interleaved"] = rng.random() < 0.4
        c["lo"] = rng.choice([1, c["hi"]])
    elif op == "read":
        c["hi"] = _log(rng, 1, 16000)
        c["B"] = _log(rng, 1, max(1, min(64, 60000 // c["hi"])))
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
    elif op == "decode":
        c["hi"] = _log(rng, 1, 4000 if small else 131072)
        c["B"] = _log(rng, 1, max(1, min(128, int(8e9) // (c["hi"] * Hkv * d * 8))))
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
    else:
        c["pre_hi"] = _log(rng, 1, 1000 if small else 131072)
        c["pre_lo"] = rng.choice([1, c["pre_hi"]])
        c["hi"] = _log(rng, 1, 300 if small else 4000)
        c["lo"] = rng.choice([1, (c["hi"] + 1) // 2, c["hi"]])
        c["B"] = _log(rng, 1, max(1, min(128, int(8e9) // ((c["pre_hi"] + 128 + c["hi"]) * Hkv * d * 8))))
        c["P"] = min(c["B"], rng.choice([1, 1, 2, 5]))
        c["alone"] = min(c["B"] - c["P"], rng.choice([0, 0, 1, 3]))
    return c


def _lengths(case):
    """(tokens per sequence the call brings or reads, tokens its cache holds before them)."""
    r = random.Random(case["mix"])
    new = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    old = [r.randint(case.get("old_lo", 0), case.get("old_hi", 0)) for _ in range(case["B"])]
    return new, old


def _groups(case):
    """Shared prefixes: (first sequence of each group and the last one's end, whole pages' keys of each)."""
    r = random.Random(case["mix"] + 1)
    last = case["B"] - case["alone"]
    cuts = sorted(r.sample(range(1, last), case["P"] - 1)) if case["P"] > 1 else []
    ps = case["page"]
    return [0, *cuts, last], [-(-r.randint(case["pre_lo"], case["pre_hi"]) // ps) * ps for _ in range(case["P"])]


def work(case):
    new, old = _lengths(case)
    Hq, Hkv, d, e = case["Hq"], case["Hkv"], case["d"], 2 if case["dtype"] == "bf16" else 4
    T, op, rows = sum(new), case["op"], case["B"] * case["Hq"] * (2 * case["d"] * e + 4)
    if op == "append":  # the rows in and out, the pages written and read back
        table = max(n + o for n, o in zip(new, old)) - min(old)
        return {"bytes": T * 2 * (Hq + 2 * Hkv) * d * e + T * 4 * Hkv * (d + 4) + min(table, T) * case["rot"] * 4,
                "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * d}
    if op == "read":
        return {"bytes": T * 2 * Hkv * (d + 4) + T * 2 * Hkv * d * e, "flops": 2 * T * Hkv * d}
    if op == "decode":
        return {"bytes": T * 2 * Hkv * (d + 4) + rows, "flops": 4 * T * Hq * d}
    cu, pre = _groups(case)
    seen = T + sum(n * (b - a) for n, a, b in zip(pre, cu, cu[1:]))
    return {"bytes": (T + sum(pre)) * 2 * Hkv * d * e + rows, "flops": 4 * seen * Hq * d}


def _quantise(y):
    """Rows [..., d] of 32-bit values -> e4m3 codes, scales [...]."""
    top = y.abs().amax(-1)
    frac, exp = torch.frexp(top)  # top = frac 2^exp, 0.5 <= frac < 1; 448 = 0.875 * 2^9
    exp = (exp - 9 + (frac > 0.875).int()).clamp_min(-126)
    scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), exp), torch.zeros_like(top))
    by = torch.where(top > 0, scale, torch.ones_like(scale))
    return (y / by[..., None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    """A user's tensors before the call: packed tokens with their offsets, the
    cache's pages with the table that says which sequence holds which."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    new, old = _lengths(case)
    B, Hq, Hkv, d, op, ps = case["B"], case["Hq"], case["Hkv"], case["d"], case["op"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def offsets(v):
        at = [0]
        for n in v:
            at.append(at[-1] + n)
        return ints(at)

    s = {"case": case, "new": new, "cu": offsets(new), "T": sum(new)}
    shared = [0] * B  # pages a sequence takes from its group's first
    if op == "shared":
        cu, pre = _groups(case)
        s["cu_prefix"], s["prefix_len"] = ints(cu), ints(pre)
        for n, a, b in zip(pre, cu, cu[1:]):
            old[a:b] = [n] * (b - a)
            shared[a + 1:b] = [n // ps] * (b - a - 1)
    s["old"] = old
    # the cache: a sequence's pages lie anywhere in it; entries past its last page are -1
    total = [n + o for n, o in zip(new, old)]
    need = [-(-n // ps) for n in total]
    num_pages = sum(need) - sum(shared) + 3
    order = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32).tolist()
    table, at = [], 0
    for n, k in zip(need, shared):
        table.append((table[-1][:k] if k else []) + order[at:at + n - k] + [-1] * (max(need) - n))
        at += n - k
    s["table"], s["kv_len"], s["keys"] = ints(table), ints(total), max(total)
    if op == "append":
        for x in ("k", "v"):
            s[x + "_cache"] = torch.zeros(num_pages, ps, Hkv, d, device=dev).to(torch.float8_e4m3fn)
            s[x + "_scale"] = torch.zeros(num_pages, Hkv, ps, device=dev)
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["q"], s["k"], s["v"] = normal(s["T"], Hq, d), normal(s["T"], Hkv, d), normal(s["T"], Hkv, d)
        return s
    for x in ("k", "v"):
        rows = normal(num_pages, ps, Hkv, d)
        if op == "shared":
            s[x + "_cache"] = rows
        else:  # rows of unequal size, as an append leaves them
            rows = rows.float().mul_(torch.rand(num_pages, ps, Hkv, 1, generator=g, device=dev).mul_(1.5).add_(0.25))
            s[x + "_cache"], scale = _quantise(rows)
            s[x + "_scale"] = scale.transpose(1, 2).contiguous()
    if op != "read":
        s["q"] = normal(B, Hq, d)
    return s


# ---- the plain forms ---------------------------------------------------------
def _slots(s):
    """(page, row within it) of every packed token, which are the last of their sequences."""
    cu, ps = s["cu"].long(), s["case"]["page"]
    t = torch.arange(s["T"], dtype=torch.int64, device=cu.device)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    pos = s["kv_len"][b].long() - cu[b + 1] + t
    return s["table"][b, pos // ps].long(), pos % ps, pos


def _plain_read(s):
    page, row, _ = _slots(s)
    dt = DTYPES[s["case"]["dtype"]]
    return tuple((s[x + "_cache"].view(torch.uint8)[page, row].view(torch.float8_e4m3fn).float() *
                  s[x + "_scale"][page, :, row][..., None]).to(dt) for x in ("k", "v"))


def _plain_append(s):
    half, page, row = s["case"]["rot"] // 2, *_slots(s)[:2]
    cs = s["rope"][_slots(s)[2]].double()[:, None]
    c, sn = cs[..., 0], cs[..., 1]

    def rotate(x):
        y = x.double()  # rounded once: a key's code depends on which side of a border it lies
        if s["case"]["interleaved"]:
            a, z = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            r = torch.stack([a * c - z * sn, z * c + a * sn], -1).flatten(-2)
        else:
            a, z = y[..., :half], y[..., half:2 * half]
            r = torch.cat([a * c - z * sn, z * c + a * sn], -1)
        return torch.cat([r, y[..., 2 * half:]], -1)

    for x, rows in (("k", rotate(s["k"]).float()), ("v", s["v"].float())):
        codes, scale = _quantise(rows)
        s[x + "_cache"].view(torch.uint8)[page, row] = codes.view(torch.uint8)
        s[x + "_scale"][page, :, row] = scale
    return rotate(s["q"]).to(s["q"].dtype), *_plain_read(s)


def _plain_decode(s):
    """Every sequence's pages spread to a padded batch [B, keys, Hkv, d], attention there."""
    at, (Hkv, d) = s["table"].clamp_min(0).long(), (s["case"]["Hkv"], s["case"]["d"])

    def keys(x):
        if s["case"]["op"] == "shared":
            y = s[x + "_cache"][at].float()
        else:
            y = s[x + "_cache"].view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
            y *= s[x + "_scale"][at].transpose(2, 3)[..., None]
        return y.flatten(1, 2)[:, :s["keys"]]

    B, Hq = s["q"].shape[:2]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    sc = torch.matmul(q, keys("k").permute(0, 2, 3, 1)) * d ** -0.5
    hidden = torch.arange(s["keys"], device=q.device)[None] >= s["kv_len"][:, None]
    sc.masked_fill_(hidden[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    out = torch.matmul(p, keys("v").transpose(1, 2)) / den
    return out.view(B, Hq, d).to(s["q"].dtype), (m + den.log()).view(B, Hq)


# ---- the library's calls -----------------------------------------------------
def _scratch(s, op, Nq, Nk):
    """The workspace a user's program allocates once for its sizes."""
    import block_sparse_long_select_gb300 as msa

    if "ws" not in s:
        c = s["case"]
        code = msa.MSA_BF16 if c["dtype"] == "bf16" else msa.MSA_FP32
        s["ws"] = msa.workspace(msa.msa_workspace_size(getattr(msa, op), c["B"], Nq, Nk, c["Hkv"], c["Hq"], c["d"], 0,
                                                       0, 0, code), s["table"].device)
    return s["ws"]


def _own_read(s):
    import block_sparse_long_select_gb300 as msa

    c = s["case"]
    one = c["lo"] == c["hi"] == 1  # one token per sequence: no offsets needed
    return msa.msa_paged_read_fp8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                  None if one else s["cu"], s["kv_len"], s["T"], dtype=DTYPES[c["dtype"]],
                                  ws=_scratch(s, "MSA_OP_PAGED_READ_FP8", s["T"], 0))


def _own_append(s):
    import block_sparse_long_select_gb300 as msa

    ws = _scratch(s, "MSA_OP_PAGED_APPEND_FP8", s["T"], 0)
    one = s["case"]["lo"] == s["case"]["hi"] == 1
    q = msa.msa_paged_append_fp8(s["q"], s["k"], s["v"], s["rope"], None if one else s["cu"], s["kv_len"], s["table"],
                                 s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                 interleaved=s["case"]["interleaved"], ws=ws)
    return q, *_own_read(s)


def _own_decode(s):
    import block_sparse_long_select_gb300 as msa

    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=s["q"].device)
    most = s["table"].shape[1] * s["case"]["page"]
    if s["case"]["op"] == "shared":
        ws = _scratch(s, "MSA_OP_FULL_DECODE_SHARED", s["case"]["P"], most)
        return msa.msa_full_attn_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_len"],
                                               s["cu_prefix"], s["prefix_len"], lse=lse, ws=ws), lse
    ws = _scratch(s, "MSA_OP_FULL_DECODE_FP8", 1, most)
    return msa.msa_full_attn_decode_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                        s["kv_len"], lse=lse, ws=ws), lse


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "read": _own_read, "decode": _own_decode, "shared": _own_decode}[op](s)
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "shared": _plain_decode}[op](s)


# ---- the definition in 64 bits, sequence by sequence and head by head -----------
def _stands_for(y):
    """What e4m3 codes with a scale per row of y (64 bits) stand for, by the grid of the format."""
    top = y.abs().amax(-1, keepdim=True)
    power = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)).clamp_min(-126)
    x = y * torch.exp2(-power)
    cell = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / cell) * cell * torch.exp2(power)


def exact(case, seed):
    s = prepare(case, seed)
    new, old, ps = s["new"], s["old"], case["page"]
    Hq, Hkv, d, op, dev = case["Hq"], case["Hkv"], case["d"], case["op"], s["table"].device
    starts = [sum(new[:b]) for b in range(case["B"])]
    if op == "append":
        half = case["rot"] // 2
        res = []
        for x in (s["q"].double(), s["k"].double()):
            for t0, n, o in zip(starts, new, old):
                cs = torch.complex(*(s["rope"][o:o + n, :, i].double() for i in (0, 1)))[:, None]
                y = x[t0:t0 + n]
                if case["interleaved"]:
                    z = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * cs
                    y[..., :2 * half] = torch.view_as_real(z).flatten(-2)
                else:
                    z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * cs
                    y[..., :half], y[..., half:2 * half] = z.real, z.imag
            res.append(x)
        return res[0], _stands_for(res[1]), _stands_for(s["v"].double())

    def cached(x, b, g):
        """Sequence b's keys or values of head g, page by page."""
        used = s["table"][b, :-(-(new[b] + old[b]) // ps)].long()
        if op == "shared":
            return s[x + "_cache"][used, :, g].reshape(-1, d)[:new[b] + old[b]].double()
        y = s[x + "_cache"].view(torch.uint8)[used, :, g].view(torch.float8_e4m3fn).double()
        return (y * s[x + "_scale"][used, g].double()[..., None]).reshape(-1, d)[:new[b] + old[b]]

    if op == "read":
        res = [torch.zeros(s["T"], Hkv, d, dtype=torch.float64, device=dev) for _ in range(2)]
        for r, x in zip(res, ("k", "v")):
            for b, (t0, n) in enumerate(zip(starts, new)):
                for g in range(Hkv):
                    r[t0:t0 + n, g] = cached(x, b, g)
        return tuple(res)
    out = torch.zeros(case["B"], Hq, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(case["B"], Hq, dtype=torch.float64, device=dev)
    for b in range(case["B"]):
        for g in range(Hkv):
            mine = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            x = s["q"][b, mine].double() @ cached("k", b, g).T / math.sqrt(d)
            lse[b, mine] = torch.logsumexp(x, 1)
            out[b, mine] = torch.softmax(x, 1) @ cached("v", b, g)
    return out, lse
