"""The serving attention operators on the sizes that they meet in use.

Three operators form one path: ``paged_kv_append`` puts rows of keys and values into the pages of a
cache, ``attention_prefill`` is the attention over whole prompts (packed sequences of different lengths,
grouped heads), and ``attention_decode`` is the attention of one new token for each sequence over the
paged cache.  Keys and values are bf16, or E4M3 codes with one fp32 scale per (token, kv head), which is
what the library's QKV projection writes.  Heads are 128 wide.

``own`` false: the operators in elementary torch operations, in fp32, rounded once at the end.
``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

HEAD_DIM = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's chat, a few hundred tokens in: the call's latency is all there is
        {"name": "decode one short fp8", "op": "decode", "cache": "fp8", "batch": 1, "shortest": 600, "longest": 600,
         "heads": 32, "kv_heads": 8, "page": 64, "lens_seed": 1},
        # a mixed batch of a server, sequences from a few tokens to thousands, small pages
        {"name": "decode ragged bf16", "op": "decode", "cache": "bf16", "batch": 24, "shortest": 5, "longest": 4096,
         "heads": 32, "kv_heads": 8, "page": 16, "lens_seed": 2},
        # a full server: the cache is streamed once for each token
        {"name": "decode full batch fp8", "op": "decode", "cache": "fp8", "batch": 64, "shortest": 2048,
         "longest": 8192, "heads": 32, "kv_heads": 8, "page": 64, "lens_seed": 3},
        # long documents, one key head for each query head
        {"name": "decode long documents bf16", "op": "decode", "cache": "bf16", "batch": 3, "shortest": 15000,
         "longest": 32768, "heads": 16, "kv_heads": 16, "page": 128, "lens_seed": 4},
        # the cache entry of one decode step, as the FP8 projection writes it
        {"name": "append step fp8", "op": "append", "rows": "fp8", "cache": "fp8", "batch": 32, "shortest": 1,
         "longest": 1, "history": 1000, "kv_heads": 8, "page": 64, "lens_seed": 5},
        # prompts of a bf16 projection into an FP8 cache, quantised on the way
        {"name": "append prompts bf16 to fp8", "op": "append", "rows": "bf16", "cache": "fp8", "batch": 9,
         "shortest": 300, "longest": 2500, "history": 0, "kv_heads": 8, "page": 64, "lens_seed": 6},
        # one short question
        {"name": "prefill one short bf16", "op": "prefill", "cache": "bf16", "batch": 1, "shortest": 77,
         "longest": 77, "heads": 32, "kv_heads": 8, "causal": True, "pad_rows": 0, "lens_seed": 7},
        # packed prompts of a server, padded to a fixed number of rows, from the FP8 projection
        {"name": "prefill packed fp8", "op": "prefill", "cache": "fp8", "batch": 24, "shortest": 20,
         "longest": 1500, "heads": 32, "kv_heads": 8, "causal": True, "pad_rows": 100, "lens_seed": 8},
        # the library's own QKV workload: 4 sequences of 2048 tokens, 32 heads each with its own keys
        {"name": "prefill 4x2048 bf16", "op": "prefill", "cache": "bf16", "batch": 4, "shortest": 2048,
         "longest": 2048, "heads": 32, "kv_heads": 32, "causal": True, "pad_rows": 0, "lens_seed": 9},
        # the same rows through the FP8 projection with grouped heads
        {"name": "prefill 4x2048 fp8", "op": "prefill", "cache": "fp8", "batch": 4, "shortest": 2048,
         "longest": 2048, "heads": 32, "kv_heads": 8, "causal": True, "pad_rows": 0, "lens_seed": 10},
        # an encoder over documents of odd lengths: no causal mask, six query heads to a key head
        {"name": "prefill full mask bf16", "op": "prefill", "cache": "bf16", "batch": 7, "shortest": 500,
         "longest": 1300, "heads": 24, "kv_heads": 4, "causal": False, "pad_rows": 0, "lens_seed": 11},
        # one long document
        {"name": "prefill long bf16", "op": "prefill", "cache": "bf16", "batch": 1, "shortest": 8192,
         "longest": 8192, "heads": 32, "kv_heads": 8, "causal": True, "pad_rows": 0, "lens_seed": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "append", "prefill", "prefill"))
    kv = rng.choice((1, 2, 4, 8, 8, 16))
    group = rng.choice((1, 2, 3, 4, 4, 5, 6, 7, 8, 8, 12, 16))
    while kv * group > 64:
        group = max(1, group // 2)
    case = {"op": op, "cache": rng.choice(("bf16", "fp8")), "kv_heads": kv, "lens_seed": rng.randrange(1 << 20)}
    if op != "append":
        case["heads"] = kv * group
    longest = _log_int(rng, 1, {"decode": 32768, "append": 4096, "prefill": 4096}[op])
    case["longest"] = longest
    case["shortest"] = max(1, _log_int(rng, 1, longest) if rng.random() < 0.7 else longest)
    batch = _log_int(rng, 1, 128)
    if op == "prefill":
        room = min(12000 // longest, int(3e8 / (case["heads"] * longest * longest)))
        case |= {"batch": max(1, min(batch, room)), "causal": rng.random() < 0.75,
                 "pad_rows": rng.choice((0, 0, 1, 33, 200))}
    elif op == "decode":
        room = int(5e8 / (longest * kv * HEAD_DIM * (2 if case["cache"] == "fp8" else 4)))
        case |= {"batch": max(1, min(batch, room)), "page": rng.choice((8, 16, 32, 64, 128))}
    else:
        case |= {"batch": max(1, min(batch, 12000 // longest)), "page": rng.choice((8, 16, 32, 64, 128)),
                 "rows": "bf16" if case["cache"] == "bf16" else rng.choice(("bf16", "fp8")),
                 "history": rng.choice((0, 1, 50, 777))}
    return case


def _lens(case):
    """The lengths of a case's sequences (new rows for an append), spread over the logarithm of the range."""
    r = random.Random(case["lens_seed"])
    lo, hi = case["shortest"], case["longest"]
    lens = [_log_int(r, lo, hi) for _ in range(case["batch"])]
    lens[r.randrange(len(lens))] = hi
    return lens


def work(case):
    lens, kv, size = _lens(case), case["kv_heads"], 1 if case["cache"] == "fp8" else 2
    rows = sum(lens)
    scales = 8 * kv if case["cache"] == "fp8" else 0  # bytes of the two scales for each token
    if case["op"] == "append":
        came = 1 if case["rows"] == "fp8" else 2
        entries = sum(-(-(n + case["history"]) // case["page"]) - case["history"] // case["page"] for n in lens)
        return {"bytes": rows * (2 * kv * HEAD_DIM * (came + size) + scales * (2 if case["rows"] == "fp8" else 1))
                + 4 * entries, "flops": 0}
    heads = case["heads"]
    if case["op"] == "decode":
        entries = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": rows * (2 * kv * HEAD_DIM * size + scales) + 4 * len(lens) * heads * HEAD_DIM + 4 * entries,
                "flops": 4 * rows * heads * HEAD_DIM}
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    return {"bytes": rows * (4 * heads * HEAD_DIM + 2 * kv * HEAD_DIM * size + scales),
            "flops": 4 * pairs * heads * HEAD_DIM}


# ---------------------------------------------------------------- inputs
def _quantise(y):
    """E4M3 codes (bytes) and scales of y [..., 128], scale = max|y| / 448 over each head of a token."""
    s = y.float().abs().amax(-1) / E4M3_MAX
    c = (y.float() / torch.where(s > 0, s, 1.0)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return c.view(torch.uint8), s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens, kv, fp8 = _lens(case), case["kv_heads"], case["cache"] == "fp8"

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    s = {"op": case["op"], "fp8": fp8, "kv": kv, "batch": len(lens)}
    if case["op"] == "prefill":
        rows, cu = sum(lens) + case["pad_rows"], [0]
        for n in lens:
            cu.append(cu[-1] + n)
        heads = case["heads"]
        s |= {"heads": heads, "causal": case["causal"], "max_len": max(lens),
              "cu": torch.tensor(cu, dtype=torch.int32, device=dev), "q": randn(rows, heads * HEAD_DIM),
              "o": torch.zeros(rows, heads * HEAD_DIM, dtype=torch.bfloat16, device=dev)}
        k, v = randn(rows, kv, HEAD_DIM), randn(rows, kv, HEAD_DIM)
        s["k_scale"] = s["v_scale"] = None
        if fp8:
            (k, s["k_scale"]), (v, s["v_scale"]) = _quantise(k), _quantise(v)
        s["k"], s["v"] = k.view(rows, -1), v.view(rows, -1)
        if own:
            import gemm_epilogue_tcgen05_gb300 as fl

            s["workspace"] = fl.attention_prefill_workspace(rows, kv, fp8, dev)
        return s

    # a cache whose pages are given out in no order
    page, before = case["page"], case.get("history", 0)
    total = [n + before for n in lens]
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
    s["kp_scale"] = s["vp_scale"] = None
    shape = (pages, kv, page, HEAD_DIM)
    if case["op"] == "append":  # an empty cache
        kind = torch.uint8 if fp8 else torch.bfloat16
        s["kp"], s["vp"] = (torch.zeros(shape, dtype=kind, device=dev) for _ in range(2))
        if fp8:
            s["kp_scale"], s["vp_scale"] = (torch.zeros(shape[:3], device=dev) for _ in range(2))
        rows, cu = sum(lens), [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = None if case["longest"] == 1 else torch.tensor(cu, dtype=torch.int32, device=dev)
        k, v = randn(rows, kv, HEAD_DIM), randn(rows, kv, HEAD_DIM)
        s["k_scale"] = s["v_scale"] = None
        if case["rows"] == "fp8":
            (k, s["k_scale"]), (v, s["v_scale"]) = _quantise(k), _quantise(v)
        s["k"], s["v"] = k.view(rows, -1), v.view(rows, -1)
        return s
    heads = case["heads"]
    s |= {"heads": heads, "q": randn(len(lens), heads * HEAD_DIM),
          "o": torch.empty(len(lens), heads * HEAD_DIM, dtype=torch.bfloat16, device=dev)}
    s["kp"], s["vp"] = randn(*shape), randn(*shape)
    if fp8:
        (s["kp"], s["kp_scale"]), (s["vp"], s["vp_scale"]) = _quantise(s["kp"]), _quantise(s["vp"])
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        s["workspace"] = fl.attention_decode_workspace(dev)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return {"append": _append, "decode": _decode, "prefill": _prefill}[s["op"]](s)


def _values(codes, scale, kind):
    """The numbers that a cache's or a projection's entries [..., 128] stand for."""
    if scale is None:
        return codes.to(kind)
    return codes.view(torch.float8_e4m3fn).to(kind) * scale[..., None].to(kind)


def _append(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        fl.paged_kv_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], cu_seqlens=s["cu"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"], k_page_scale=s["kp_scale"],
                           v_page_scale=s["vp_scale"])
    else:
        rows, kv, page = s["k"].shape[0], s["kv"], s["page"]
        row = torch.arange(rows, device=s["k"].device)
        if s["cu"] is None:
            seq, pos = row, s["lens"].long() - 1
        else:
            seq = torch.searchsorted(s["cu"].long(), row, right=True) - 1
            pos = s["lens"].long()[seq] - s["cu"].long()[seq + 1] + row
        at, slot = s["table"].long()[seq, pos // page], pos % page
        k, v = s["k"].view(rows, kv, HEAD_DIM), s["v"].view(rows, kv, HEAD_DIM)
        ks, vs = s["k_scale"], s["v_scale"]
        if s["fp8"]:
            if ks is None:
                (k, ks), (v, vs) = _quantise(k), _quantise(v)
            s["kp_scale"][at, :, slot], s["vp_scale"][at, :, slot] = ks, vs
        s["kp"][at, :, slot], s["vp"][at, :, slot] = k, v
    if s["fp8"]:
        return [s["kp"].view(torch.float8_e4m3fn), s["vp"].view(torch.float8_e4m3fn), s["kp_scale"], s["vp_scale"]]
    return [s["kp"], s["vp"]]


def _decode(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        return fl.attention_decode(s["q"], s["kp"], s["vp"], s["table"], s["lens"], k_page_scale=s["kp_scale"],
                                   v_page_scale=s["vp_scale"], O=s["o"], workspace=s["workspace"])
    b, kv = s["batch"], s["kv"]
    at = s["table"].long()

    def dense(pages, scale):  # [batch, kv heads, tokens, 128]
        x = _values(pages[at], None if scale is None else scale[at], torch.float32)
        return x.transpose(1, 2).reshape(b, kv, -1, HEAD_DIM)

    k, v = dense(s["kp"], s["kp_scale"]), dense(s["vp"], s["vp_scale"])
    q = s["q"].float().view(b, kv, -1, HEAD_DIM)
    x = torch.matmul(q, k.transpose(2, 3)) * HEAD_DIM ** -0.5
    there = torch.arange(x.shape[-1], device=x.device) < s["lens"][:, None, None, None]
    x = x.masked_fill(~there, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.reshape(b, -1).to(torch.bfloat16)


def _prefill(s):
    if own:
        import gemm_epilogue_tcgen05_gb300 as fl

        return fl.attention_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["cu"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"], causal=s["causal"], O=s["o"], workspace=s["workspace"])
    b, kv, n, rows = s["batch"], s["kv"], s["max_len"], s["q"].shape[0]
    cu = s["cu"].long()
    pos = torch.arange(n, device=cu.device)
    there = pos[None] < (cu[1:] - cu[:-1])[:, None]  # [batch, n]
    at = torch.where(there, cu[:-1, None] + pos[None], 0)

    def padded(x, scale):  # [batch, kv heads, n, 128]
        x = x.view(rows, kv, HEAD_DIM)[at]
        return _values(x, None if scale is None else scale[at], torch.float32).transpose(1, 2)

    k, v = padded(s["k"], s["k_scale"]), padded(s["v"], s["v_scale"])
    q = s["q"].view(rows, kv, -1, HEAD_DIM)[at].float().permute(0, 2, 3, 1, 4)  # [batch, kv heads, group, n, 128]
    x = torch.matmul(q, k.transpose(2, 3)[:, :, None]) * HEAD_DIM ** -0.5
    seen = there[:, None, :].expand(b, n, n)
    if s["causal"]:
        seen = seen & (pos[None, :] <= pos[:, None])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    o = torch.matmul(p, v[:, :, None]) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, -1)
    s["o"][at[there]] = o[there].to(torch.bfloat16)
    return s["o"]


# ---------------------------------------------------------------- the definition in 64 bits
def _attend(q, k, v, causal):
    """softmax(q k^T / sqrt(128)) v of one kv head: q [group, n, 128], k and v [tokens, 128], all fp64."""
    out, n = torch.empty_like(q), k.shape[0]
    for first in range(0, q.shape[1], 2048):
        part = q[:, first:first + 2048]
        x = part @ k.T / math.sqrt(HEAD_DIM)
        if causal:
            i = torch.arange(first, first + part.shape[1], device=k.device)
            x.masked_fill_(torch.arange(n, device=k.device)[None] > i[:, None], -math.inf)
        out[:, first:first + 2048] = torch.softmax(x, -1) @ v
    return out


def _nearest_e4m3(x):
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    lens, kv = _lens(case), case["kv_heads"]
    if case["op"] == "append":
        kp, vp = (torch.zeros(s["kp"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
        out = [kp, vp]
        if s["fp8"]:
            out += [torch.zeros(kp.shape[:3], dtype=torch.float64, device="cuda") for _ in range(2)]
        first = 0
        for b, n in enumerate(lens):
            pos = torch.arange(case["history"], case["history"] + n, device="cuda")
            page, slot = s["table"][b].long()[pos // case["page"]], pos % case["page"]
            for i, (x, scale) in enumerate(((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))):
                x = x[first:first + n].view(n, kv, HEAD_DIM)
                if s["fp8"] and scale is None:
                    x = x.double()
                    sc = x.abs().amax(-1) / E4M3_MAX
                    x = _nearest_e4m3(x / sc.clamp_min(1e-300)[..., None])
                elif s["fp8"]:
                    x, sc = x.view(torch.float8_e4m3fn).double(), scale[first:first + n].double()
                out[i][page, :, slot] = x.double()
                if s["fp8"]:
                    out[2 + i][page, :, slot] = sc
            first += n
        return out
    heads = case["heads"]
    group = heads // kv
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for b, n in enumerate(lens):
        if case["op"] == "decode":
            page, slot = s["table"][b].long()[torch.arange(n, device="cuda") // case["page"]], torch.arange(n, device="cuda") % case["page"]
            k = _values(s["kp"][page, :, slot], None if s["kp_scale"] is None else s["kp_scale"][page, :, slot], torch.float64)
            v = _values(s["vp"][page, :, slot], None if s["vp_scale"] is None else s["vp_scale"][page, :, slot], torch.float64)
            q, rows = s["q"][b:b + 1], slice(b, b + 1)
        else:
            rows = slice(first, first + n)
            k, v = (_values(s[x][rows].view(n, kv, HEAD_DIM), None if s[x + "_scale"] is None else s[x + "_scale"][rows],
                            torch.float64) for x in ("k", "v"))
            q = s["q"][rows]
            first += n
        q = q.double().view(-1, heads, HEAD_DIM).transpose(0, 1)
        for h in range(kv):
            mine = slice(h * group, (h + 1) * group)
            part = _attend(q[mine], k[:, h], v[:, h], case["op"] == "prefill" and case["causal"])
            o.view(-1, heads, HEAD_DIM)[rows, mine] = part.transpose(0, 1)
    return o
