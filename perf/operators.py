"""Workloads of the paged key/value cache: appending new tokens to it (with the
position rotation) and the attention of the new tokens over it, each in a
plain form of elementary torch operations and through the library."""
import math
import random

import torch

own = False

_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_ROPE_BASE = 500000.0


def _case(name, op, seqs, new, past, q_heads, kv_heads, head_dim, page, cache, ragged=0, mixed=0, interleaved=0, pick=1):
    return {"name": name, "op": op, "seqs": seqs, "new": new, "past": past, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "cache": cache, "ragged": ragged, "mixed": mixed,
            "interleaved": interleaved, "pick": pick}


def listed():
    return [
        # one decoding step of a small batch: the call's latency
        _case("append_step_16", "append", 16, 1, 2000, 32, 8, 128, 16, "bf16", ragged=1),
        # a whole prompt of the 8192-token attention layer into an FP8 cache
        _case("append_prompt_8192", "append", 1, 8192, 0, 32, 8, 128, 64, "e4m3"),
        # ragged chunks of several requests, small heads, rotation of neighbouring pairs
        _case("append_chunks_7", "append", 7, 1501, 700, 16, 4, 64, 32, "e5m2", ragged=1, interleaved=1),
        # a large prefill batch: 32768 tokens of one layer's cache
        _case("append_batch_32768", "append", 8, 4096, 1000, 32, 8, 128, 64, "bf16"),
        # one request, one token, a short cache: the call's latency
        _case("decode_1x500", "attention", 1, 1, 500, 32, 8, 128, 16, "bf16"),
        # an ordinary decoding batch of unequal requests
        _case("decode_64x8000", "attention", 64, 1, 8000, 32, 8, 128, 64, "bf16", ragged=1),
        # long requests on an FP8 cache
        _case("decode_16x65536_e4m3", "attention", 16, 1, 65536, 32, 8, 128, 64, "e4m3"),
        # one very long request: the work has to be split over its keys
        _case("decode_1x524287", "attention", 1, 1, 524287, 32, 8, 128, 128, "bf16"),
        # drafted tokens of a batch checked in one pass
        _case("drafts_32x5", "attention", 32, 5, 4001, 32, 8, 128, 32, "e4m3", ragged=1),
        # a prompt attended from an empty cache
        _case("prompt_8192", "attention", 1, 8192, 0, 32, 8, 128, 64, "bf16"),
        # one chunk of a long prompt on an FP8 cache
        _case("chunk_2048_of_32768_e4m3", "attention", 1, 2048, 30720, 32, 8, 128, 64, "e4m3"),
        # single tokens and chunks together, small heads
        _case("mixed_24x700", "attention", 24, 700, 5000, 24, 8, 64, 64, "bf16", ragged=1, mixed=1),
    ]


def _spread(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v + (v == 3072)))


def draw(rng):
    op = rng.choice(["append", "attention", "attention"])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    c = _case("", op, 1, 1, 0, kv_heads * group, kv_heads, rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]),
              rng.choice(["bf16", "bf16", "e4m3", "e4m3", "e5m2"]), interleaved=rng.randrange(2), pick=rng.randrange(1 << 20))
    del c["name"]
    kind = rng.choice(["steps", "drafts", "chunks", "mixed"])
    if op == "append":
        c["seqs"] = _spread(rng, 1, 256)
        c["new"] = 1 if kind == "steps" else _spread(rng, 2, max(2, 32768 // c["seqs"]))
        c["past"] = _spread(rng, 1, 2000)
        c["ragged"], c["mixed"] = rng.randrange(2), int(kind == "mixed")
        return c
    if kind == "steps":
        c["seqs"] = _spread(rng, 1, 128)
        c["past"] = _spread(rng, 200, min(400000, (1 << 20) // c["seqs"]))
    elif kind == "drafts":
        c["seqs"], c["new"] = _spread(rng, 1, 48), rng.randrange(2, 9)
        c["past"] = _spread(rng, 100, min(60000, 300000 // c["seqs"]))
    else:
        c["seqs"] = _spread(rng, 1, 24) if kind == "mixed" else _spread(rng, 1, 6)
        c["new"] = _spread(rng, 9, 5000 // c["seqs"] if kind == "chunks" else 600)
        c["past"] = _spread(rng, 1, min(40000, 60000000 // (c["seqs"] * c["new"]))) if kind == "chunks" else _spread(rng, 50, 5000)
        c["mixed"] = int(kind == "mixed")
    c["ragged"] = rng.randrange(2)
    return c


def _lengths(case):
    """(new tokens, cached tokens) of every sequence, from the case alone."""
    r = random.Random(case["pick"])
    out = []
    for b in range(case["seqs"]):
        new = r.randint((case["new"] + 1) // 2, case["new"]) if case["ragged"] else case["new"]
        past = r.randint(case["past"] // 8, case["past"]) if case["ragged"] else case["past"]
        out.append((1 if case["mixed"] and b % 2 == 0 else new, past))
    return out


def work(case):
    lens, D, Hq, Hkv = _lengths(case), case["head_dim"], case["q_heads"], case["kv_heads"]
    esz = 2 if case["cache"] == "bf16" else 1
    T = sum(n for n, _ in lens)
    if case["op"] == "append":
        rows = min(T, max(n + p for n, p in lens))      # table rows that are read
        return {"bytes": T * ((2 * Hq + 2 * Hkv) * D * 2 + 2 * Hkv * D * esz) + rows * D * 4,
                "flops": T * (Hq + Hkv) * D * 3}
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in lens)
    kv = sum(n + p for n, p in lens)
    return {"bytes": 2 * kv * Hkv * D * esz + T * Hq * (2 * D * 2 + 4), "flops": 4 * D * Hq * pairs}


class _State:
    pass


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    s = _State()
    s.case = case
    lens, D, Hq, Hkv, page = _lengths(case), case["head_dim"], case["q_heads"], case["kv_heads"], case["page"]
    T = sum(n for n, _ in lens)
    s.max_new, s.max_kv = max(n for n, _ in lens), max(n + p for n, p in lens)
    # q, k, v side by side, as the fused projection leaves them; the attention alone has its rotated queries in hand
    if case["op"] == "append":
        qkv = normal(T, (Hq + 2 * Hkv) * D)
        s.q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s.k = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s.v = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    else:
        s.q = normal(T, Hq, D).mul_(2.0)
    ints = dict(dtype=torch.int32, device="cuda")
    s.q_offsets = torch.tensor([0] + [n for n, _ in lens], **ints).cumsum(0, dtype=torch.int32)
    s.kv_lens = torch.tensor([n + p for n, p in lens], **ints)
    # every sequence's pages lie scattered over the pool
    need = [-(-(n + p) // page) for n, p in lens]
    pool = sum(need) + max(1, sum(need) // 8)
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(max(need), device="cuda")
    s.page_table = torch.where(col < (at[1:] - at[:-1])[:, None], order[(at[:-1, None] + col).clamp(max=pool - 1)], 0).contiguous()
    shape = (pool, Hkv, page, D)
    s.k_scale = s.v_scale = None
    if case["cache"] == "bf16":
        s.k_pages, s.v_pages = normal(*shape), normal(*shape)
    else:   # scales as the calibration leaves them: amax / fmax
        kind, fmax = _FP8[case["cache"]], _FMAX[case["cache"]]
        s.k_scale = torch.full((1,), 6.0 / fmax, device="cuda")
        s.v_scale = torch.full((1,), 5.5 / fmax, device="cuda")
        s.k_pages = (normal(*shape).float() / s.k_scale).clamp_(-fmax, fmax).to(kind)
        s.v_pages = (normal(*shape).float() / s.v_scale).clamp_(-fmax, fmax).to(kind)
    if case["op"] == "append":
        freq = _ROPE_BASE ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        angle = torch.arange(s.max_kv, device="cuda", dtype=torch.float64)[:, None] * freq
        s.rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        s.q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    else:
        s.out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s.lse = torch.empty((T, Hq), device="cuda")
    if own:
        import fp8_fine_grained_x128_gb300 as fg
        s.cache = fg.PagedKV(s.k_pages, s.v_pages, s.k_scale, s.v_scale)
        s.batch = fg.PagedBatch(s.q_offsets, s.kv_lens, s.page_table, s.max_new)
        if case["op"] == "attention":
            s.workspace = fg.new_attention_workspace()
    return s


def _tokens(s):
    """Sequence and position of every new token."""
    t = torch.arange(s.q.shape[0], device="cuda")
    seq = torch.searchsorted(s.q_offsets, t, right=True) - 1
    return seq, s.kv_lens[seq] - s.q_offsets[seq + 1] + t


def _rotate(x, cos, sin, interleaved):
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(s):
    case, half = s.case, s.case["head_dim"] // 2
    seq, pos = _tokens(s)
    cos, sin = s.rope[pos, :half], s.rope[pos, half:]
    q = _rotate(s.q.float(), cos, sin, case["interleaved"])
    k = _rotate(s.k.float(), cos, sin, case["interleaved"])
    v = s.v.float()
    where = s.page_table[seq, pos // case["page"]], pos % case["page"]
    if case["cache"] == "bf16":
        raw, k, v = torch.int16, k.bfloat16(), v.bfloat16()
    else:
        kind, fmax = _FP8[case["cache"]], _FMAX[case["cache"]]
        raw = torch.uint8
        k, v = (k / s.k_scale).clamp(-fmax, fmax).to(kind), (v / s.v_scale).clamp(-fmax, fmax).to(kind)
    s.k_pages.view(raw)[where[0], :, where[1]] = k.view(raw)
    s.v_pages.view(raw)[where[0], :, where[1]] = v.view(raw)
    return q.bfloat16(), s.k_pages, s.v_pages


def _gathered(s, pages, scale):
    """[seqs, kv heads, keys, head_dim] in 32 bits, through the page table."""
    table = s.page_table.long()
    x = pages.view(torch.int16 if pages.element_size() == 2 else torch.uint8)[table].view(pages.dtype).float()
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :s.max_kv]
    return x if scale is None else x * scale


def _attention_plain(s):
    case = s.case
    B, D, Hq, Hkv = case["seqs"], case["head_dim"], case["q_heads"], case["kv_heads"]
    k, v = _gathered(s, s.k_pages, s.k_scale), _gathered(s, s.v_pages, s.v_scale)
    seq, pos = _tokens(s)
    row = torch.arange(s.q.shape[0], device="cuda") - s.q_offsets[seq]
    q = torch.zeros((B, s.max_new, Hq, D), device="cuda")
    q[seq, row] = s.q.float()
    at = torch.full((B, s.max_new), -1, device="cuda")
    at[seq, row] = pos.to(at.dtype)
    q = q.view(B, s.max_new, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    score = q @ k.transpose(-1, -2) * D ** -0.5
    score = score.view(B, Hq, s.max_new, s.max_kv)
    score.masked_fill_(torch.arange(s.max_kv, device="cuda") > at[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    out = (p.view(B, Hkv, -1, s.max_kv) @ v).view(B, Hq, s.max_new, D)
    out = out / torch.where(total == 0, 1.0, total)[..., None]
    lse = total.log() + top[..., 0]
    return out.transpose(1, 2)[seq, row].bfloat16(), lse.transpose(1, 2)[seq, row]


def run(state):
    s, case = state, state.case
    if not own:
        return _append_plain(s) if case["op"] == "append" else _attention_plain(s)
    import fp8_fine_grained_x128_gb300 as fg
    if case["op"] == "append":
        fg.rope_append_kv(s.cache, s.batch, s.k, s.v, s.rope, q=s.q, q_out=s.q_out, interleaved=bool(case["interleaved"]))
        return s.q_out, s.k_pages, s.v_pages
    fg.paged_attention(s.cache, s.batch, s.q, s.out, s.workspace, lse=s.lse)
    return s.out, s.lse


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    D, Hq, Hkv, page = case["head_dim"], case["q_heads"], case["kv_heads"], case["page"]
    G, lens = Hq // Hkv, _lengths(case)
    pages_of, start = s.page_table.long(), 0
    if case["op"] == "append":
        kp, vp = s.k_pages.double(), s.v_pages.double()
        qs, half = [], D // 2
        freq = _ROPE_BASE ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        fmax = _FMAX.get(case["cache"], math.inf)
        ks, vs = (1.0, 1.0) if s.k_scale is None else (s.k_scale.double(), s.v_scale.double())
        for b, (n, p) in enumerate(lens):
            at = torch.arange(p, p + n, device="cuda")
            turn = torch.polar(torch.ones((n, half), dtype=torch.float64, device="cuda"), at[:, None] * freq)[:, None]

            def turned(x):
                x = x.double()
                z = torch.complex(x[..., 0::2], x[..., 1::2]) if case["interleaved"] else torch.complex(x[..., :half], x[..., half:])
                z = z * turn
                return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)

            qs.append(turned(s.q[start:start + n]))
            pg, r = pages_of[b, at // page], at % page
            kp[pg, :, r] = (turned(s.k[start:start + n]) / ks).clamp(-fmax, fmax)
            vp[pg, :, r] = (s.v[start:start + n].double() / vs).clamp(-fmax, fmax)
            start += n
        return torch.cat(qs), kp, vp
    out = torch.zeros((s.q.shape[0], Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((s.q.shape[0], Hq), -math.inf, dtype=torch.float64, device="cuda")
    ks, vs = (1.0, 1.0) if s.k_scale is None else (s.k_scale.double(), s.v_scale.double())
    raw = torch.int16 if case["cache"] == "bf16" else torch.uint8
    for b, (n, p) in enumerate(lens):
        L = n + p
        mine = pages_of[b, :-(-L // page)]
        seen = torch.arange(L, device="cuda") <= torch.arange(p, L, device="cuda")[:, None]
        for h in range(Hkv):
            k = (s.k_pages.view(raw)[mine, h].view(s.k_pages.dtype).double() * ks).reshape(-1, D)[:L]
            v = (s.v_pages.view(raw)[mine, h].view(s.v_pages.dtype).double() * vs).reshape(-1, D)[:L]
            for j in range(h * G, (h + 1) * G):
                a = (s.q[start:start + n, j].double() @ k.T) / math.sqrt(D)
                a = a.masked_fill(~seen, -math.inf)
                lse[start:start + n, j] = torch.logsumexp(a, -1)
                out[start:start + n, j] = torch.softmax(a, -1) @ v
        start += n
    return out, lse
