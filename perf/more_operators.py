"""Serving operators: a cache held in 4 bits, attention with a sliding window, on the sizes they meet in use.

Four operators form one path.  ``paged_kv_append_int4`` quantises rows of keys and values into the pages of a cache:
codes of 4 bits, one scale for each 32 values.  ``paged_kv_read`` gives cached tokens back as rows, what a new part
of a prompt attends to.  ``attention_decode_window`` is the attention of one new token for each sequence over a paged
cache (bf16, E4M3 or 4 bits), ``attention_prefill_window`` that of a prompt, or of its next part behind what is
already there; both see the last `window` tokens and the first `sinks` ones (a window of 0: all of them).  Heads are
128 wide.

The 4-bit cache: s = max|y| / 7 over 32 consecutive values of a head, rounded to five significant bits (nearest even),
codes = y / s rounded to the nearest even whole number, in [-7, 7], so that code * s is a bf16 number.  Values of a
group whose largest magnitude is below 2^-120 become zero, s too; a group with a value that is not finite has a NaN
for s.  Codes lie two to a byte, the even column in the low half.

``own`` false: the operators in elementary torch operations, in fp32, rounded once at the end.
``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

HEAD_DIM = 128
GROUP = 32  # values that share a scale
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat, a few hundred tokens in: the call's latency is all there is
        {"name": "decode one short int4", "op": "decode", "cache": "int4", "batch": 1, "shortest": 600, "longest": 600,
         "heads": 32, "kv_heads": 8, "page": 64, "window": 0, "sinks": 0, "lens_seed": 1},
        # a mixed batch of a server, from a few tokens to long chats, layers that look at the last 1024 tokens
        {"name": "decode ragged window int4", "op": "decode", "cache": "int4", "batch": 24, "shortest": 5,
         "longest": 32768, "heads": 32, "kv_heads": 8, "page": 16, "window": 1024, "sinks": 4, "lens_seed": 2},
        # a full server: the cache is streamed once for each token
        {"name": "decode full batch int4", "op": "decode", "cache": "int4", "batch": 64, "shortest": 2048,
         "longest": 8192, "heads": 32, "kv_heads": 8, "page": 64, "window": 0, "sinks": 0, "lens_seed": 3},
        # long documents in a bf16 cache, a window of 4096 and a system prompt's head that stays visible
        {"name": "decode long window bf16", "op": "decode", "cache": "bf16", "batch": 16, "shortest": 8192,
         "longest": 65536, "heads": 16, "kv_heads": 16, "page": 128, "window": 4096, "sinks": 64, "lens_seed": 4},
        # one decode step of a layer: the new token into the cache, then its attention
        {"name": "step int4", "op": "step", "cache": "int4", "batch": 32, "shortest": 1, "longest": 4096, "heads": 32,
         "kv_heads": 8, "page": 64, "window": 0, "sinks": 0, "lens_seed": 5},
        # prompts of a bf16 projection into the cache, and back as the rows that their attention takes
        {"name": "append prompts int4", "op": "append", "cache": "int4", "batch": 9, "shortest": 300, "longest": 2500,
         "history": 0, "kv_heads": 8, "page": 64, "lens_seed": 6},
        # the next 512 tokens of a long prompt, and the whole context for their attention
        {"name": "append chunk int4", "op": "append", "cache": "int4", "batch": 1, "shortest": 512, "longest": 512,
         "history": 8000, "kv_heads": 8, "page": 64, "lens_seed": 7},
        # a prefix that was cached for an earlier request
        {"name": "read prefix int4", "op": "read", "cache": "int4", "batch": 1, "shortest": 32768, "longest": 32768,
         "kv_heads": 8, "page": 64, "lens_seed": 8},
        # the ends of 24 contexts of an FP8 cache with small pages
        {"name": "read ragged fp8", "op": "read", "cache": "fp8", "batch": 24, "shortest": 20, "longest": 1500,
         "kv_heads": 8, "page": 16, "lens_seed": 9},
        # one long document in a layer with a window of 1024
        {"name": "prefill window long bf16", "op": "prefill", "cache": "bf16", "batch": 1, "shortest": 8192,
         "longest": 8192, "heads": 32, "kv_heads": 8, "window": 1024, "sinks": 4, "history": 0, "pad_rows": 0,
         "lens_seed": 10},
        # packed prompts of a server, padded to a fixed number of rows, from the FP8 projection, a short window
        {"name": "prefill window packed fp8", "op": "prefill", "cache": "fp8", "batch": 24, "shortest": 20,
         "longest": 1500, "heads": 32, "kv_heads": 8, "window": 256, "sinks": 4, "history": 0, "pad_rows": 100,
         "lens_seed": 11},
        # the next parts of six prompts behind up to 4000 tokens that are already there, no window
        {"name": "prefill chunks bf16", "op": "prefill", "cache": "bf16", "batch": 6, "shortest": 33, "longest": 512,
         "heads": 32, "kv_heads": 8, "window": 0, "sinks": 0, "history": 4000, "pad_rows": 0, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "step", "append", "read", "prefill", "prefill"))
    kv = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice((1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16))
    while kv * group > 64:
        group = max(1, group // 2)
    kinds = {"decode": ("int4", "int4", "fp8", "bf16"), "step": ("int4",), "append": ("int4",),
             "read": ("int4", "fp8", "bf16"), "prefill": ("bf16", "fp8")}[op]
    case = {"op": op, "cache": rng.choice(kinds), "kv_heads": kv, "lens_seed": rng.randrange(1 << 20)}
    longest = _log_int(rng, 1, {"decode": 32768, "step": 16384, "append": 4096, "read": 16384, "prefill": 4096}[op])
    case["longest"] = longest
    case["shortest"] = max(1, _log_int(rng, 1, longest) if rng.random() < 0.7 else longest)
    batch = _log_int(rng, 1, 128)
    if op in ("decode", "step", "prefill"):
        case |= {"heads": kv * group, "window": 0, "sinks": 0}
        if rng.random() < 0.6:
            case |= {"window": _log_int(rng, 1, 8192), "sinks": rng.choice((0, 0, 1, 4, 16, 64, 130))}
    if op == "prefill":
        case["history"] = rng.choice((0, 0, 1, 100, 2000))
        n = longest + case["history"]
        room = min(12000 // n, int(1.5e8 / (case["heads"] * longest * n)))
        return case | {"batch": max(1, min(batch, room)), "pad_rows": rng.choice((0, 0, 1, 33, 200))}
    case["page"] = rng.choice((8, 16, 32, 64, 128))
    if op == "append":
        case["history"] = rng.choice((0, 0, 1, 50, 777, 5000))
        return case | {"batch": max(1, min(batch, 12000 // (longest + case["history"])))}
    if op == "read":
        return case | {"batch": max(1, min(batch, 24000 // longest))}
    return case | {"batch": max(1, min(batch, int(5e8 / (longest * kv * HEAD_DIM * 4))))}


def _lens(case):
    """The lengths of a case's sequences (new rows where there is a history), spread over the logarithm of the range."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["shortest"], case["longest"]
    lens = [_log_int(r, lo, hi) for _ in range(case["batch"])]
    lens[r.randrange(len(lens))] = hi
    return lens


def _history(case):
    """What each sequence has in front of its new rows: up to `history` tokens, the first sequence all of them."""
    r = random.Random(case["lens_seed"] + 1)
    most = case.get("history", 0)
    return [most if b == 0 or most == 0 else r.randrange(most + 1) for b in range(case["batch"])]


def _seen(n, case):
    """How many of its first n tokens the last of them sees."""
    return min(n, case["window"] + case["sinks"]) if case["window"] else n


def work(case):
    lens, kv = _lens(case), case["kv_heads"]
    token = 2 * kv * {"bf16": 2 * HEAD_DIM, "fp8": HEAD_DIM + 4, "int4": HEAD_DIM // 2 + 2 * HEAD_DIM // GROUP}[case["cache"]]
    row, entry = 2 * kv * 2 * HEAD_DIM, 4  # bytes of a token's keys and values as bf16 rows; of a page table's entry
    if case["op"] in ("append", "read"):
        total = [n + h for n, h in zip(lens, _history(case))]
        entries = sum(-(-n // case["page"]) for n in total)
        if case["op"] == "read":
            return {"bytes": sum(lens) * (token + row) + entry * entries, "flops": 0}
        # new rows in, their codes out; then the cache in, the whole context out
        return {"bytes": sum(lens) * (row + token) + sum(total) * (token + row) + entry * entries, "flops": 0}
    heads = case["heads"]
    if case["op"] in ("decode", "step"):
        seen = [_seen(n, case) for n in lens]
        entries = sum(-(-n // case["page"]) for n in seen)
        new = len(lens) * (row + token) if case["op"] == "step" else 0
        return {"bytes": sum(seen) * token + 4 * len(lens) * heads * HEAD_DIM + entry * entries + new,
                "flops": 4 * sum(seen) * heads * HEAD_DIM}
    w, sinks = case["window"], case["sinks"]

    def pairs_up_to(n):  # of queries 0 .. n - 1 with all the keys that they see
        full = min(n, w + sinks) if w else n
        return full * (full + 1) // 2 + (n - full) * (w + sinks)

    keys = pairs = 0
    for n, h in zip(lens, _history(case)):
        pairs += pairs_up_to(n + h) - pairs_up_to(h)
        keys += n + h if w == 0 else min(n + h, n + w - 1 + sinks)
    return {"bytes": sum(lens) * 4 * heads * HEAD_DIM + keys * token, "flops": 4 * pairs * heads * HEAD_DIM}


# ---------------------------------------------------------------- inputs
def _quantise(y):
    """E4M3 codes (bytes) and scales of y [..., 128], scale = max|y| / 448 over each head of a token."""
    s = y.float().abs().amax(-1) / E4M3_MAX
    c = (y.float() / torch.where(s > 0, s, 1.0)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return c.view(torch.uint8), s


def _quantise_int4(y):
    """Packed codes (bytes [..., 64]) and scales (bf16 [..., 4]) of y [..., 128], one scale for 32 values."""
    y = y.float().unflatten(-1, (-1, GROUP))
    a = y.abs().amax(-1)
    bits = (a / 7.0).view(torch.int32)
    s = (((bits + 0x3FFFF + ((bits >> 19) & 1)) >> 19) << 19).view(torch.float32)  # five significant bits
    s = torch.where(a < 2.0 ** -120, torch.zeros_like(s), s)
    c = torch.round(y / torch.where(s > 0, s, 1.0)[..., None]).clamp(-7, 7)
    fine = torch.isfinite(a)
    s = torch.where(fine, s, math.nan)
    c = torch.where((fine & (s > 0))[..., None], c, 0.0).to(torch.int32).flatten(-2)
    return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8), s.to(torch.bfloat16)


def _values(codes, scale, kind, cache):
    """The numbers [..., 128] that a cache's or a projection's entries stand for."""
    if cache == "bf16":
        return codes.to(kind)
    if cache == "fp8":
        return codes.view(torch.float8_e4m3fn).to(kind) * scale[..., None].to(kind)
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    c = ((n ^ 8) - 8).to(kind).unflatten(-1, (-1, GROUP))
    return (c * scale[..., None].to(kind)).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, history, kv, cache = _lens(case), _history(case), case["kv_heads"], case["cache"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    def offsets(counts):
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        return torch.tensor(cu, dtype=torch.int32, device=dev)

    total = [n + h for n, h in zip(lens, history)]
    s = {"op": case["op"], "cache": cache, "kv": kv, "batch": len(lens), "window": case.get("window", 0),
         "sinks": case.get("sinks", 0), "longest": max(total), "ks": None, "vs": None}
    if case["op"] == "prefill":
        rows, k_rows, heads = sum(lens) + case["pad_rows"], sum(total) + case["pad_rows"], case["heads"]
        s |= {"heads": heads, "longest_new": max(lens), "cu": offsets(lens),
              "cu_k": offsets(total) if case["history"] else None, "q": randn(rows, heads * HEAD_DIM),
              "o": torch.zeros(rows, heads * HEAD_DIM, dtype=torch.bfloat16, device=dev)}
        k, v = randn(k_rows, kv, HEAD_DIM), randn(k_rows, kv, HEAD_DIM)
        if cache == "fp8":
            (k, s["ks"]), (v, s["vs"]) = _quantise(k), _quantise(v)
        s["k"], s["v"] = k.view(k_rows, -1), v.view(k_rows, -1)
        if own:
            import gemm_epilogue_tcgen05_gb300 as fl

            s["workspace"] = fl.attention_prefill_workspace(k_rows, kv, cache == "fp8", dev)
        return s

    # a cache whose pages are given out in no order
    page = case["page"]
    need = [-(-n // page) for n in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    width, at, starts = max(need), 0, []
    for n in need:
        starts.append(at)
        at += n
    col = torch.arange(width, device=dev)
    at = torch.tensor(starts, device=dev)[:, None] + torch.minimum(col[None], torch.tensor(need, device=dev)[:, None] - 1)
    s |= {"table": order[at].contiguous(), "lens": torch.tensor(total, dtype=torch.int32, device=dev), "page": page}
    s["kp"], s["vp"] = randn(pages, kv, page, HEAD_DIM), randn(pages, kv, page, HEAD_DIM)
    if cache != "bf16":
        quantise = _quantise if cache == "fp8" else _quantise_int4
        (s["kp"], s["ks"]), (s["vp"], s["vs"]) = quantise(s["kp"]), quantise(s["vp"])
    if case["op"] in ("append", "step"):  # the rows that come in, and their place
        rows = sum(lens) if case["op"] == "append" else len(lens)
        s["k_new"], s["v_new"] = randn(rows, kv * HEAD_DIM), randn(rows, kv * HEAD_DIM)
        s["cu"] = offsets(lens) if case["op"] == "append" else None
    if case["op"] in ("append", "read"):  # the rows that are read back
        s["cu_read"], s["rows"] = offsets(total), sum(total)
        s["k"], s["v"] = (torch.empty(sum(total), kv * HEAD_DIM, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return s
    heads = case["heads"]
    s |= {"heads": heads, "q": randn(len(lens), heads * HEAD_DIM),
          "o": torch.empty(len(lens), heads * HEAD_DIM, dtype=torch.bfloat16, device=dev)}
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        s["workspace"] = fl.attention_decode_workspace(dev)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if s["op"] == "prefill":
        return _prefill(s)
    if s["op"] == "decode":
        return _decode(s)
    if s["op"] == "read":
        return _read(s)
    _append(s)
    if s["op"] == "append":  # what 4 bits hold is given as the values that they stand for: read back
        return _read(s) + [s["ks"], s["vs"]]
    return [_decode(s), s["ks"], s["vs"]]


def _append(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        fl.paged_kv_append_int4(s["k_new"], s["v_new"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"],
                                cu_seqlens=s["cu"])
        return
    rows, kv, page = s["k_new"].shape[0], s["kv"], s["page"]
    row = torch.arange(rows, device=s["k_new"].device)
    if s["cu"] is None:
        seq, pos = row, s["lens"].long() - 1
    else:
        seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
        pos = s["lens"].long()[seq] - s["cu"].long()[seq + 1] + row
    at, slot = s["table"].long()[seq, pos // page], pos % page
    (k, ks), (v, vs) = (_quantise_int4(s[x].view(rows, kv, HEAD_DIM)) for x in ("k_new", "v_new"))
    s["kp"][at, :, slot], s["vp"][at, :, slot], s["ks"][at, :, slot], s["vs"][at, :, slot] = k, v, ks, vs


def _read(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        k, v = fl.paged_kv_read(s["kp"], s["vp"], s["table"], s["lens"], cu_seqlens=s["cu_read"],
                                k_page_scale=s["ks"], v_page_scale=s["vs"], K=s["k"], V=s["v"])
        return [k, v]
    row = torch.arange(s["rows"], device=s["kp"].device)
    cu, page = s["cu_read"].long(), s["page"]
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["lens"].long()[seq] - cu[seq + 1] + row
    at, slot = s["table"].long()[seq, pos // page], pos % page

    def rows_of(pages, scale):
        x = _values(pages[at, :, slot], None if scale is None else scale[at, :, slot], torch.float32, s["cache"])
        return x.to(torch.bfloat16).view(s["rows"], -1)

    return [rows_of(s["kp"], s["ks"]), rows_of(s["vp"], s["vs"])]


def _visible(query, key, window, sinks):
    """Which keys (positions) a query (position) sees."""
    seen = key <= query
    if window:
        seen = seen & ((key > query - window) | (key < sinks))
    return seen


def _decode(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        return fl.attention_decode_window(s["q"], s["kp"], s["vp"], s["table"], s["lens"], window=s["window"],
                                          sinks=s["sinks"], k_page_scale=s["ks"], v_page_scale=s["vs"], O=s["o"],
                                          workspace=s["workspace"])
    b, kv = s["batch"], s["kv"]
    at = s["table"].long()

    def dense(pages, scale):  # [batch, kv heads, tokens, 128]
        x = _values(pages[at], None if scale is None else scale[at], torch.float32, s["cache"])
        return x.transpose(1, 2).reshape(b, kv, -1, HEAD_DIM)

    k = dense(s["kp"], s["ks"])
    q = s["q"].float().view(b, kv, -1, HEAD_DIM)
    x = torch.matmul(q, k.transpose(2, 3)) * HEAD_DIM ** -0.5
    seen = _visible(s["lens"].long()[:, None] - 1, torch.arange(x.shape[-1], device=x.device), s["window"], s["sinks"])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, dense(s["vp"], s["vs"])) / p.sum(-1, keepdim=True)
    return o.reshape(b, -1).to(torch.bfloat16)


def _prefill(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        return fl.attention_prefill_window(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], cu_seqlens_k=s["cu_k"],
                                           window=s["window"], sinks=s["sinks"], k_scale=s["ks"], v_scale=s["vs"],
                                           O=s["o"], workspace=s["workspace"])
    b, kv, n, rows = s["batch"], s["kv"], s["longest_new"], s["q"].shape[0]
    cu = s["cu"].long()
    cu_k = cu if s["cu_k"] is None else s["cu_k"].long()
    new, total = cu[1:] - cu[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(n, device=cu.device), torch.arange(s["longest"], device=cu.device)
    mine, theirs = i < new[:, None], j < total[:, None]  # [batch, n], [batch, keys]
    at, at_k = torch.where(mine, cu[:-1, None] + i, 0), torch.where(theirs, cu_k[:-1, None] + j, 0)

    def padded(x, scale):  # [batch, kv heads, keys, 128]
        x = x.view(x.shape[0], kv, -1)[at_k]
        return _values(x, None if scale is None else scale[at_k], torch.float32, s["cache"]).transpose(1, 2)

    k, v = padded(s["k"], s["ks"]), padded(s["v"], s["vs"])
    q = s["q"].view(rows, kv, -1, HEAD_DIM)[at].float().permute(0, 2, 3, 1, 4)  # [batch, kv heads, group, n, 128]
    x = torch.matmul(q, k.transpose(2, 3)[:, :, None]) * HEAD_DIM ** -0.5
    pos = (total - new)[:, None] + i  # of each query
    seen = theirs[:, None, :] & _visible(pos[:, :, None], j, s["window"], s["sinks"])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    o = torch.matmul(p, v[:, :, None]) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, -1)
    s["o"][at[mine]] = o[mine].to(torch.bfloat16)
    return s["o"]


# ---------------------------------------------------------------- the definition in 64 bits
def _numbers(codes, scale):
    """What entries of a cache or of rows stand for, [..., 128] in 64 bits."""
    if scale is None:
        return codes.double()
    if codes.shape[-1] == HEAD_DIM:
        return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]
    low, high = codes.long() % 16, codes.long() // 16
    n = torch.empty(*codes.shape[:-1], HEAD_DIM, dtype=torch.float64, device=codes.device)
    n[..., 0::2], n[..., 1::2] = low, high
    return torch.where(n > 7, n - 16, n) * scale.double().repeat_interleave(GROUP, -1)


def _int4_of(y):
    """The numbers, and the scales, that 4 bits hold of y [..., 128]."""
    y = y.double().view(*y.shape[:-1], HEAD_DIM // GROUP, GROUP)
    most = y.abs().max(-1).values
    part, power = torch.frexp(most.clamp_min(2.0 ** -120) / 7)  # part in [1/2, 1)
    s = torch.ldexp(torch.round(part * 32), power - 5).to(torch.bfloat16).double()  # a power of two may be an ulp off
    s = s * (most >= 2.0 ** -120)
    c = torch.round(y / s.clamp_min(1e-300)[..., None]) * (s > 0)[..., None]
    return (c * s[..., None]).flatten(-2), s


def _attend(q, k, v, window, sinks):
    """q [heads, n, 128] are the last n tokens of k and v [tokens, 128] (fp64), each seeing what its position sees."""
    out, n, keys = torch.empty_like(q), q.shape[1], k.shape[0]
    j = torch.arange(keys, device=k.device)[None]
    for first in range(0, n, 2048):
        part = q[:, first:first + 2048]
        i = torch.arange(first, first + part.shape[1], device=k.device)[:, None] + (keys - n)
        hidden = j > i
        if window:
            hidden = hidden | ((j + window <= i) & (j >= sinks))
        x = (part @ k.T / math.sqrt(HEAD_DIM)).masked_fill_(hidden, -math.inf)
        out[:, first:first + 2048] = torch.softmax(x, -1) @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    lens, history, kv, dev = _lens(case), _history(case), case["kv_heads"], "cuda"
    if case["op"] != "prefill":
        at = [(s["table"][b].long()[torch.arange(n + h, device=dev) // s["page"]],
               torch.arange(n + h, device=dev) % s["page"]) for b, (n, h) in enumerate(zip(lens, history))]

    cached = {}  # of each sequence: its keys and values [tokens, kv heads, 128]
    for x, scale in (("k", "ks"), ("v", "vs")):
        if case["op"] == "prefill":
            break
        pages, scales = s[x + "p"], s[scale]
        cached[x] = [_numbers(pages[page, :, slot], None if scales is None else scales[page, :, slot])
                     for page, slot in at]
        if case["op"] in ("append", "step"):
            held, first = s[scale].double(), 0
            for b, n in enumerate(lens):
                n = n if case["op"] == "append" else 1
                new, new_scale = _int4_of(s[x + "_new"][first:first + n].view(n, kv, HEAD_DIM))
                cached[x][b][-n:] = new
                page, slot = at[b]
                held[page[-n:], :, slot[-n:]] = new_scale
                first += n
            cached[scale] = held
    if case["op"] in ("read", "append"):
        rows = [torch.cat(cached[x]).flatten(1) for x in ("k", "v")]
        return rows + [cached["ks"], cached["vs"]] if case["op"] == "append" else rows

    heads = case["heads"]
    group = heads // kv
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=dev)
    first = first_k = 0
    for b, (n, h) in enumerate(zip(lens, history)):
        if case["op"] == "prefill":
            rows, keys = slice(first, first + n), slice(first_k, first_k + n + h)
            k, v = (_numbers(s[x][keys].view(n + h, kv, HEAD_DIM), None if s[y] is None else s[y][keys])
                    for x, y in (("k", "ks"), ("v", "vs")))
            first, first_k = first + n, first_k + n + h
        else:
            rows, k, v = slice(b, b + 1), cached["k"][b], cached["v"][b]
        q = s["q"][rows].double().view(-1, heads, HEAD_DIM).transpose(0, 1)
        for g in range(kv):
            mine = slice(g * group, (g + 1) * group)
            part = _attend(q[mine], k[:, g], v[:, g], case["window"], case["sinks"])
            o.view(-1, heads, HEAD_DIM)[rows, mine] = part.transpose(0, 1)
    return [o, cached["ks"], cached["vs"]] if case["op"] == "step" else o
