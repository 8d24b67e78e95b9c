"""The attention side of a serving step around the MoE layer, as measured cases.

Three operators work on one paged key/value cache held in NVFP4 (packed E2M1
codes, an E4M3 scale per 16 elements, an fp32 scale per kv head):

  norm   per-head RMS norms of queries and keys with the position rotation, in
         one pass that also writes the keys and values into the cache
  attn   attention of ragged batches (single tokens, chunks, mixtures) over
         the cache
  pages  forking sequences, freeing them, and compacting the cache's pages

A page record of one kv head holds, for `page` tokens, key codes, key scales,
value codes, value scales, one after the other: page * D * 9 / 8 bytes.  The
pool of one layer is uint8 [pages, Hkv, page * D * 9 / 8].

`run` computes the operators in elementary torch operations in fp32, or (where
`own` is set) through the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one conversation: latency
        dict(name="norm_one", op="norm", T=1, Hq=64, Hkv=4, D=128, rot=128, pairs=False),
        # an odd chunk of a smaller model with a partial, interleaved rotation
        dict(name="norm_chunk", op="norm", T=1777, Hq=20, Hkv=5, D=64, rot=32, pairs=True),
        # a full prefill batch
        dict(name="norm_prefill", op="norm", T=16384, Hq=64, Hkv=4, D=128, rot=128, pairs=False),
        # one user in a short conversation: latency
        dict(name="attn_one", op="attn", B=1, q=1, kv=700, Hq=64, Hkv=4, D=128, window=0, ragged=False),
        # a full decode batch with contexts of all lengths
        dict(name="attn_decode", op="attn", B=256, q=1, kv=8192, Hq=64, Hkv=4, D=128, window=0, ragged=True),
        # two very long contexts: few rows, the cache has to be split
        dict(name="attn_long", op="attn", B=2, q=1, kv=131072, Hq=64, Hkv=4, D=128, window=0, ragged=True),
        # a long prompt's later chunk
        dict(name="attn_prefill", op="attn", B=1, q=4096, kv=12289, Hq=64, Hkv=4, D=128, window=0, ragged=False),
        # several prompts' chunks of unequal lengths, sliding window, small heads
        dict(name="attn_chunks", op="attn", B=13, q=700, kv=5000, Hq=40, Hkv=8, D=64, window=1024, ragged=True),
        # one beam split in two: latency
        dict(name="pages_fork_few", op="pages", kind="fork", S=8, n=2, layers=4, kv=900, pages=256, Hkv=4, D=128),
        # parallel samples of many prompts, all layers
        dict(name="pages_fork_many", op="pages", kind="fork", S=256, n=128, layers=32, kv=1500, pages=2500, Hkv=4, D=128),
        # a batch of finished sequences with shared prefixes
        dict(name="pages_free", op="pages", kind="free", S=512, n=400, layers=1, kv=6000, pages=20000, Hkv=1, D=64),
        # a fragmented pool squeezed together, all layers
        dict(name="pages_compact", op="pages", kind="compact", S=128, n=64, layers=32, kv=1500, pages=2500, Hkv=4, D=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "attn", "attn", "pages"))
    D = rng.choice((64, 128, 128))
    Hkv = rng.choice((1, 2, 4, 8))
    if op == "norm":
        pairs = rng.random() < 0.3
        rot = rng.choice((32, D // 2, D))
        Hq = Hkv * rng.randint(1, 64 // Hkv)
        return dict(op="norm", T=_spread(rng, 1, 16384), Hq=Hq, Hkv=min(Hkv, 4), D=D, rot=rot, pairs=pairs)
    if op == "attn":
        Hq = Hkv * rng.randint(1, min(16, 64 // Hkv))
        window = rng.choice((0, 0, 0, _spread(rng, 100, 4000)))
        if rng.random() < 0.6:  # decode, a few tokens each at most
            q = rng.choice((1, 1, 1, 2, 4))
            kv = _spread(rng, 16, 60000)
            B = _spread(rng, 1, max(1, min(256, 1_000_000 // (kv * Hkv))))
        else:
            q = _spread(rng, 16, 4000)
            kv = q + _spread(rng, 1, 8000)
            B = _spread(rng, 1, max(1, min(16, 2_000_000_000 // (q * kv * Hq))))
        return dict(op="attn", B=B, q=q, kv=kv, Hq=Hq, Hkv=Hkv, D=D, window=window, ragged=rng.random() < 0.7)
    kind = rng.choice(("fork", "free", "compact"))
    S = _spread(rng, 4, 256)
    kv = _spread(rng, 100, 1500)
    return dict(op="pages", kind=kind, S=S, n=max(1, S // rng.choice((2, 3, 4))), layers=rng.choice((1, 3, 8, 24)),
                kv=kv, pages=S * (kv // PAGE + 1) + rng.randint(50, 300), Hkv=min(Hkv, 4), D=D)


# ------------------------------------------------------------ lengths of a case
def _lens(c):
    """(new tokens, context with them) of every sequence, as a scheduler has them on the host: the case's own."""
    g = torch.Generator().manual_seed(c["B"] * 7919 + c["kv"])
    B, q, kv = c["B"], c["q"], c["kv"]
    if not c["ragged"]:
        return [q] * B, [kv] * B
    f = torch.rand(2, B, generator=g).tolist()
    qs = [q if q <= 4 else max(1, int(q * x)) for x in f[0]]
    kvs = [max(n, int(kv * (0.1 + 0.9 * x))) for n, x in zip(qs, f[1])]
    qs[-1], kvs[-1] = q, kv  # work() and memory go by the longest
    return qs, kvs


def _mean_pairs(c):
    """Visible (query, key) pairs and keys read of one head, of the lengths that _lens draws."""
    qs, kvs = _lens(c)
    pairs = keys = 0
    for n, L in zip(qs, kvs):
        W = c["window"] if c["window"] > 0 else L
        full = min(n, max(0, n - (W - (L - n))) if L - n < W else n)  # queries that see W keys
        rest = n - full                                              # queries that see all up to themselves
        pairs += full * min(W, L) + sum(range(L - n + 1, L - n + rest + 1))
        keys += min(L, W + n - 1)
    return pairs, keys


def work(case):
    c = case
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "norm":
        T, Hq = c["T"], c["Hq"]
        n = T * (Hq + Hkv) * D
        return dict(bytes=T * D * (4 * Hq + 4 * Hkv + 1.125 * Hkv) + T * (4 * c["rot"] + 12) + 4 * D, flops=10 * n)
    if c["op"] == "attn":
        qs, _ = _lens(c)
        pairs, keys = _mean_pairs(c)
        return dict(bytes=keys * Hkv * D * 1.125 + sum(qs) * c["Hq"] * D * 4, flops=4 * D * c["Hq"] * pairs)
    record = Hkv * PAGE * D * 9 // 8
    M = -(-c["kv"] // PAGE) + 1
    small = 8 * c["pages"] + 8 * c["S"] * (M + 1)
    if c["kind"] == "free":
        return dict(bytes=small, flops=0)
    moved = c["n"] if c["kind"] == "fork" else _moved(c)
    return dict(bytes=small + 2 * moved * c["layers"] * record, flops=0)


def _moved(c):
    """Pages that compacting has to move (of the state that prepare makes with seed 0)."""
    refs = _tables(c, 0)[2]
    live = int((refs > 0).sum())
    return int((refs[live:] > 0).sum())


# ------------------------------------------------------------------- the state
def _quantise(x, g):
    """fp32 [..., D] and g broadcastable to [..., 1] -> (codes uint8 [..., D/2], scale bytes uint8 [..., D/16])."""
    b = x.unflatten(-1, (-1, 16))
    g = g.unsqueeze(-1)
    s = (b.abs().amax(-1, keepdim=True) / (g * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * g
    a = torch.where(d == 0, torch.zeros_like(b), b.abs() / torch.where(d == 0, torch.ones_like(d), d))
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
            + (a >= 3.5).byte() + (a > 5.0).byte())
    code = (code + torch.signbit(b).byte() * 8).flatten(-2)
    return code[..., 0::2] + code[..., 1::2] * 16, s.squeeze(-1).view(torch.uint8)


def _sections(pool, D):
    """Views of a pool [..., Hkv, record]: key codes, key scales, value codes, value scales, each [..., Hkv, page, bytes]."""
    P = pool.shape[-1] * 8 // (9 * D)
    a, b = P * D // 2, P * D // 16
    kc, ks, vc, vs = pool.split((a, b, a, b), -1)
    return [t.unflatten(-1, (P, -1)) for t in (kc, ks, vc, vs)]


def _tables(c, seed):
    """Block table, lengths and page counts of a pool in use: rows share their first pages in pairs, pages lie scattered."""
    g = torch.Generator().manual_seed(seed * 104729 + 5)
    S, n, N = c["S"], c["n"], c["pages"]
    M = -(-c["kv"] // PAGE) + 1
    lens = (c["kv"] * (0.3 + 0.7 * torch.rand(S, generator=g))).int().clamp(min=1)
    if c["kind"] == "fork":
        lens[S - n:] = 0  # empty rows that the forks go to
    used = -(-lens // PAGE)
    j = torch.arange(M).unsqueeze(0)
    mine = j < used.unsqueeze(1)
    # odd rows share the first third of the full pages of the row before them
    share = torch.minimum(lens // PAGE, torch.roll(lens, 1, 0) // PAGE) // 3
    share[0::2] = 0
    shared = j < share.unsqueeze(1)
    order = torch.randperm(N, generator=g).int()
    new = mine & ~shared
    at = (new.flatten().cumsum(0) - 1).view(S, M)
    table = torch.where(new, order[at.clamp(0, N - 1)], torch.full((S, M), -1, dtype=torch.int32))
    table = torch.where(shared, torch.roll(table, 1, 0), table)
    if c["kind"] == "compact":  # sequences that have ended leave holes
        gone = torch.randperm(S, generator=g)[:n]
        table[gone], lens[gone] = -1, 0
    refs = torch.bincount(table[table >= 0].long(), minlength=N).int()
    return table, lens, refs


def prepare(case, seed):
    c = case
    gen = torch.Generator(DEV).manual_seed(seed)
    D, Hkv = c["D"], c["Hkv"]
    record = PAGE * D * 9 // 8
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    if c["op"] == "pages":
        table, lens, refs = (t.to(DEV) for t in _tables(c, seed))
        pool = torch.randint(0, 256, (c["layers"], c["pages"], Hkv, record), generator=gen, device=DEV, dtype=torch.uint8)
        s = dict(c=c, pool=pool, table=table, lens=lens, refs=refs)
        if c["kind"] == "fork":
            s["src"] = torch.randint(0, c["S"] - c["n"], (c["n"],), generator=gen, device=DEV, dtype=torch.int32)
            s["dst"] = torch.arange(c["S"] - c["n"], c["S"], device=DEV, dtype=torch.int32)
        elif c["kind"] == "free":
            s["rows"] = torch.randperm(c["S"], generator=gen, device=DEV)[:c["n"]].int()
        return s
    gk = 0.002 + 0.0005 * torch.rand(Hkv, generator=gen, device=DEV)
    gv = 0.002 + 0.0005 * torch.rand(Hkv, generator=gen, device=DEV)
    if c["op"] == "norm":
        T, Hq = c["T"], c["Hq"]
        # queries, keys and values are slices of one projection's output
        qkv = randn(T, (Hq + 2 * Hkv) * D).mul_(1.5).bfloat16()
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
        top = 40960
        inv = 1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(top, device=DEV, dtype=torch.float64).unsqueeze(1) * inv
        pages = T // PAGE + 3
        first = int(torch.randint(0, top - T, (1,), generator=torch.Generator().manual_seed(seed)))
        order = torch.randperm(pages, generator=gen, device=DEV)
        t = torch.arange(T, device=DEV) + first % PAGE
        return dict(c=c, q=q, k=k, v=v, wq=(1 + 0.1 * randn(D)).bfloat16(), wk=(1 + 0.1 * randn(D)).bfloat16(),
                    cos_sin=torch.cat((ang.cos(), ang.sin()), 1).float(), gk=gk, gv=gv,
                    pos=torch.arange(first, first + T, device=DEV, dtype=torch.int32),
                    slots=order[t // PAGE] * PAGE + t % PAGE,
                    pool=torch.zeros(pages, Hkv, record, dtype=torch.uint8, device=DEV))
    qs, kvs = _lens(c)
    T, B, M = sum(qs), c["B"], -(-max(kvs) // PAGE)
    used = torch.tensor([-(-L // PAGE) for L in kvs])
    N = int(used.sum()) + 5
    # bytes that nobody has written yet are anything; here they decode to NaN
    pool = torch.full((N, Hkv, record), 0xFF, dtype=torch.uint8, device=DEV)
    kc, ks, vc, vs = _sections(pool, D)
    loud = 1 + 3 * (torch.rand(Hkv, 1, D, generator=gen, device=DEV) > 0.97)  # some channels of the keys stand out
    for a in range(0, N, 1024):
        m = min(N, a + 1024) - a
        kc[a:a + m], ks[a:a + m] = _quantise(randn(m, Hkv, PAGE, D) * loud, gk.view(-1, 1, 1))
        vc[a:a + m], vs[a:a + m] = _quantise(randn(m, Hkv, PAGE, D), gv.view(-1, 1, 1))
    mine = torch.arange(M).unsqueeze(0) < used.unsqueeze(1)
    table = torch.full((B, M), -1, dtype=torch.int32, device=DEV)
    table[mine.to(DEV)] = torch.randperm(N, generator=gen, device=DEV)[:int(used.sum())].int()
    last = torch.tensor([L % PAGE for L in kvs], device=DEV)
    tail = table[torch.arange(B, device=DEV), (used - 1).to(DEV)].long()
    past = (last.unsqueeze(1) > 0) & (torch.arange(PAGE, device=DEV) >= last.unsqueeze(1))
    i, off = past.nonzero(as_tuple=True)
    ks[tail[i], :, off] = 0xFF
    vs[tail[i], :, off] = 0xFF
    start = torch.tensor([0] + qs).cumsum(0)
    return dict(c=c, q=(1.7 * randn(T, c["Hq"], D)).bfloat16(), pool=pool, gk=gk, gv=gv, table=table,
                starts=start.int().to(DEV), lens=torch.tensor(kvs, dtype=torch.int32, device=DEV), max_q=max(qs),
                scale=D ** -0.5)


# -------------------------------------------------------------- plain operators
def _tree_sum(x):
    """Sum over the last axis (a power of two), neighbours first: the order that makes the cache's bytes reproducible."""
    return x if x.shape[-1] == 1 else _tree_sum(x[..., 0::2] + x[..., 1::2])


def _norm_rope(x, w, eps, cos, sin, rot, pairs):
    x = x.float()
    r = 1.0 / torch.sqrt(_tree_sum(x * x) * (1.0 / x.shape[-1]) + eps)
    x = x * r * w.float()
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    c, s = cos.unsqueeze(1), sin.unsqueeze(1)
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_norm(s):
    c = s["c"]
    D, rot = c["D"], c["rot"]
    cos, sin = s["cos_sin"][s["pos"].long()].split(rot // 2, 1)
    q = _norm_rope(s["q"], s["wq"], 1e-6, cos, sin, rot, c["pairs"])
    k = _norm_rope(s["k"], s["wk"], 1e-6, cos, sin, rot, c["pairs"])
    kc, ks, vc, vs = _sections(s["pool"], D)
    page, off = s["slots"] // PAGE, s["slots"] % PAGE
    kc[page, :, off], ks[page, :, off] = _quantise(k, s["gk"].view(-1, 1))
    vc[page, :, off], vs[page, :, off] = _quantise(s["v"].float(), s["gv"].view(-1, 1))
    return q.bfloat16(), s["pool"]


def _decoded(codes, scales, g):
    """[..., page, bytes] -> fp32 [..., page, D]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    x = lut[x.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return x.flatten(-2) * g


def _plain_attn(s):
    c, q, table = s["c"], s["q"], s["table"]
    D, Hkv, G = c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    B, M = table.shape
    parts = [t.movedim(1, 0).contiguous() for t in _sections(s["pool"], D)]  # [Hkv, pages, page, bytes]
    at = table.clamp(min=0).long()
    K = _decoded(parts[0][:, at], parts[1][:, at], s["gk"].view(-1, 1, 1, 1, 1)).flatten(2, 3)  # [Hkv, B, keys, D]
    V = _decoded(parts[2][:, at], parts[3][:, at], s["gv"].view(-1, 1, 1, 1, 1)).flatten(2, 3)
    i = torch.arange(s["max_q"], device=DEV)
    n = s["starts"].diff()
    row = (s["starts"][:-1].unsqueeze(1) + i).clamp(max=q.shape[0] - 1).long()  # [B, max_q]
    place = (s["lens"] - n).unsqueeze(1) + i  # position of each query in its context
    key = torch.arange(M * PAGE, device=DEV)
    there = key < s["lens"].unsqueeze(1)  # [B, keys]
    K = torch.where(there.unsqueeze(-1), K, 0.0)
    V = torch.where(there.unsqueeze(-1), V, 0.0)
    seen = (key <= place.unsqueeze(-1)) & there.unsqueeze(1)
    if c["window"] > 0:
        seen = seen & (key > place.unsqueeze(-1) - c["window"])
    Q = q[row].float().unflatten(2, (Hkv, G)).permute(2, 0, 1, 3, 4)  # [Hkv, B, max_q, G, D]
    S = torch.matmul(Q.flatten(2, 3), K.transpose(-1, -2)).unflatten(2, (-1, G)) * s["scale"]
    S = torch.where(seen.unsqueeze(2), S, -math.inf)
    S -= S.amax(-1, keepdim=True).clamp(min=-1e30)
    S = S.exp_()
    l = S.sum(-1)
    out = torch.matmul(S.flatten(2, 3), V).unflatten(2, (-1, G)) / torch.where(l > 0, l, 1.0).unsqueeze(-1)
    return out.permute(1, 2, 0, 3, 4)[(i < n.unsqueeze(1))].flatten(1, 2).bfloat16()  # [T, Hq, D]


def _plain_fork(s):
    pool, src, dst = s["pool"], s["src"].long(), s["dst"].long()
    table, lens, refs = s["table"].clone(), s["lens"].clone(), s["refs"].clone()
    rows, L = table[src], lens[src].long()
    partial = L % PAGE > 0
    new = torch.argsort((refs != 0).byte(), stable=True)[(partial.cumsum(0) - 1).clamp(min=0)].int()
    j = torch.arange(table.shape[1], device=DEV)
    full = j < (L // PAGE).unsqueeze(1)
    last = partial.unsqueeze(1) & (j == (L // PAGE).unsqueeze(1))
    refs += torch.bincount(rows[full].long(), minlength=refs.numel()).int()
    refs[new[partial].long()] = 1
    pool[:, new[partial].long()] = pool[:, rows[last].long()]
    table[dst] = torch.where(last, new.unsqueeze(1), torch.where(full, rows, -1))
    lens[dst] = L.int()
    return table, lens, refs, pool


def _plain_free(s):
    table, lens, refs, rows = s["table"].clone(), s["lens"].clone(), s["refs"].clone(), s["rows"].long()
    t = table[rows]
    refs -= torch.bincount(t[t >= 0].long(), minlength=refs.numel()).int()
    table[rows] = -1
    lens[rows] = 0
    return table, lens, refs


def _plain_compact(s):
    pool, refs, table = s["pool"], s["refs"], s["table"]
    live = refs > 0
    n = live.sum()
    i = torch.arange(refs.numel(), device=DEV)
    hole, high = (~live & (i < n)).nonzero().flatten(), (live & (i >= n)).nonzero().flatten()
    remap = torch.where(live, i, -1).int()
    remap[high] = hole.int()
    pool[:, hole] = pool[:, high]
    new = torch.zeros_like(refs)
    new[remap[live].long()] = refs[live]
    return torch.where(table >= 0, remap[table.clamp(min=0).long()], -1), new, remap, pool


PLAIN = dict(norm=_plain_norm, attn=_plain_attn, fork=_plain_fork, free=_plain_free, compact=_plain_compact)


def run(state):
    s, c = state, state["c"]
    op = c["kind"] if c["op"] == "pages" else c["op"]
    if not own:
        return PLAIN[op](s)
    import mixture_experts_layer_fwd_gb300 as moe
    if op == "norm":
        q, _ = moe.moe_qk_norm_rope(s["q"], s["k"], s["cos_sin"], s["pos"], wq=s["wq"], wk=s["wk"], eps=1e-6,
                                    interleaved=c["pairs"], v=s["v"], pool=s["pool"], g_k=s["gk"], g_v=s["gv"],
                                    slots=s["slots"])
        return q, s["pool"]
    if op == "attn":
        return moe.moe_kv4_attention(s["q"], s["pool"], s["gk"], s["gv"], s["starts"], s["lens"], s["table"],
                                     scale=s["scale"], window=c["window"])
    if op == "fork":
        o = moe.moe_kv_fork(s["src"], s["dst"], s["table"], s["lens"], s["refs"], s["pool"], page_size=PAGE)
        return o["table"], o["lens"], o["refs"], s["pool"]
    if op == "free":
        o = moe.moe_kv_free(s["rows"], s["table"], s["lens"], s["refs"], page_size=PAGE)
        return o["table"], o["lens"], o["refs"]
    o = moe.moe_kv_compact(s["table"], s["refs"], s["pool"])
    return o["table"], o["refs"], o["remap"], s["pool"]


# ------------------------------------------------------------------ in 64 bits
def _value(nibble):
    """E2M1 by its definition: sign, two exponent bits (bias 1), one mantissa bit."""
    e, m = (nibble >> 1) & 3, (nibble & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()))
    return torch.where(nibble >= 8, -v, v)


def _scale(b):
    """E4M3 by its definition (bias 7, three mantissa bits)."""
    e, m = (b >> 3) & 15, (b & 7).double()
    return torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7)) * torch.where(b >= 128, -1.0, 1.0)


def _read(record, first, D, n, g):
    """n tokens of one head's page records [pages, bytes], from byte `first` of a record on, in 64 bits."""
    P = record.shape[1] * 8 // (9 * D)
    codes = record[:, first:first + P * D // 2].reshape(-1, D // 2)[:n].int()
    scales = record[:, first + P * D // 2:first + P * D * 9 // 16].reshape(-1, D // 16)[:n].int()
    x = torch.empty(codes.shape[0], D, dtype=torch.float64, device=codes.device)
    x[:, 0::2], x[:, 1::2] = _value(codes & 15), _value(codes >> 4)
    return x * _scale(scales).repeat_interleave(16, 1) * g.double()


def exact(case, seed):
    c = case
    if c["op"] == "pages":
        return None  # whole numbers only
    s = prepare(case, seed)
    D = c["D"]
    if c["op"] == "norm":
        x, w = s["q"].double(), s["wq"].double()
        x = x / (x.square().mean(2, keepdim=True) + 1e-6).sqrt() * w
        cos, sin = s["cos_sin"].double()[s["pos"].long()].unsqueeze(1).chunk(2, 2)
        h = c["rot"] // 2
        i = 2 * torch.arange(h, device=DEV) if c["pairs"] else torch.arange(h, device=DEV)
        j = i + 1 if c["pairs"] else i + h
        y = x.clone()
        y[:, :, i] = x[:, :, i] * cos - x[:, :, j] * sin
        y[:, :, j] = x[:, :, j] * cos + x[:, :, i] * sin
        return y, None  # the cache holds codes
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    start, lens = s["starts"].tolist(), s["lens"].tolist()
    for b in range(c["B"]):
        n, L = start[b + 1] - start[b], lens[b]
        pages = s["table"][b, :-(-L // PAGE)].long()
        p = torch.arange(L - n, L, device=DEV).unsqueeze(1)
        t = torch.arange(L, device=DEV)
        seen = (t <= p) & ((t > p - c["window"]) if c["window"] > 0 else (t >= 0))
        for h in range(c["Hkv"]):
            rec = s["pool"][pages, h]
            K = _read(rec, 0, D, L, s["gk"][h])
            V = _read(rec, PAGE * D * 9 // 16, D, L, s["gv"][h])
            for a in range(h * G, h * G + G):
                z = (s["q"][start[b]:start[b + 1], a].double() @ K.T * s["scale"]).masked_fill(~seen, -math.inf)
                out[start[b]:start[b + 1], a] = torch.softmax(z, 1) @ V
    return out
