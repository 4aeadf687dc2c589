"""The paged 3-bit KV cache, measured: appending tokens, page management, and
decode attention over pages of which a batch may share a prefix.

A page holds 64 tokens. For one layer a cache is `pages`, uint8
[n_pages x H x block], where the block of a (page, head) is, with rb = 3 D / 8
bytes a row of 3-bit codes:

  K codes   64 rows of rb bytes, one per token
  V codes   16 groups of 4 tokens, [group][byte of the row][token of the group]
  K scales  fp32 [64];  V scales  fp32 [64]

A token may be kept at 4 bits: its K scale then has the sign bit set, byte 0
of its K row says which of the page's 4-bit rows is its own, and
`codes4` [n_pages x H x rows4 x D] holds that row (D / 2 bytes of K, then of V).

Sequences are rows of `tables` (page ids), `lens` (tokens) and `refs` (how
many table entries name a page; 0 = free).
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's new tokens of 64 sequences, heads of a LLaMA-7B-shaped layer
        dict(name="append decode 64", op="append", n=64, H=32, Hq=32, D=128, decode=True, rows4=0),
        # the prompt of one sequence, bos at 4 bits
        dict(name="append prompt 4096", op="append", n=4096, H=32, Hq=32, D=128, decode=False, rows4=1),
        # an odd prompt with few small heads, part of the batch padding
        dict(name="append odd 777", op="append", n=777, H=5, Hq=10, D=64, decode=False, rows4=0),
        # one step of a small beam search: the beams are freed, forked again and grown by a token
        dict(name="beams 2x4", op="beams", P=2, C=4, longest=300, L=2, H=4, D=128, rows4=0),
        # the same for 16 requests of 4 beams over all layers of a model
        dict(name="beams 16x4 32 layers", op="beams", P=16, C=4, longest=700, L=32, H=8, D=128, rows4=1),
        # pages moved in all layers at once
        dict(name="copy 300 pages", op="copy", n=300, n_pages=700, L=32, H=8, D=128, rows4=0),
        # a short sequence alone: what a call costs
        dict(name="attention 1x129", op="attention", B=1, Sq=1, H=32, G=1, D=128, shared=0, longest=129, rows4=0, ragged=False),
        # a few requests behind one prompt
        dict(name="attention 8 on 4096", op="attention", B=8, Sq=1, H=32, G=1, D=128, shared=64, longest=257, rows4=1, ragged=True),
        # a full batch behind one prompt, heads as in a LLaMA-7B-shaped layer
        dict(name="attention 64 on 4096", op="attention", B=64, Sq=1, H=32, G=1, D=128, shared=64, longest=512, rows4=0, ragged=True),
        # grouped heads and a long shared document
        dict(name="attention 96 on 32768", op="attention", B=96, Sq=1, H=8, G=4, D=128, shared=512, longest=300, rows4=0, ragged=True),
        # no shared prefix: every sequence its own pages
        dict(name="attention 64x4096", op="attention", B=64, Sq=1, H=32, G=1, D=128, shared=0, longest=4096, rows4=0, ragged=True),
        # drafted tokens verified together, wide heads, 4-bit tokens
        dict(name="attention 5 drafts", op="attention", B=5, Sq=4, H=4, G=2, D=256, shared=10, longest=1000, rows4=2, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "beams", "copy", "attention", "attention", "attention"])
    D = rng.choice([64, 128, 128, 256])
    rows4 = rng.choice([0, 0, 1, 3])
    if op == "append":
        H = _log(rng, 1, 32)
        decode = rng.random() < 0.5
        n = _log(rng, 1, 512 if decode else 4096 * 32 * 128 // (32 * D))
        return dict(op=op, n=n, H=H, Hq=H * rng.choice([1, 2, 4]), D=D, decode=decode, rows4=rows4)
    if op == "beams":
        return dict(op=op, P=_log(rng, 1, 16), C=rng.randint(1, 4), longest=_log(rng, 1, 700), L=_log(rng, 1, 16),
                    H=_log(rng, 1, 8), D=D, rows4=rows4)
    if op == "copy":
        n = _log(rng, 1, 300)
        return dict(op=op, n=n, n_pages=2 * n + rng.randint(0, 60), L=_log(rng, 1, 15), H=_log(rng, 1, 8), D=D, rows4=rows4)
    G = rng.choice([1, 1, 2, 4, 8])
    H = _log(rng, 1, 16)
    Sq = rng.choice([1, 1, 1, 2, 5])
    B = _log(rng, 1, 96)
    shared = rng.choice([0, _log(rng, 1, 256)])
    longest = _log(rng, 1, 2048)
    c = dict(op="attention", B=B, Sq=Sq, H=H, G=G, D=D, shared=shared, longest=longest, rows4=rows4, ragged=True)
    while work(c)["flops"] > 4e10:  # no more than the largest listed one
        c["shared"], c["longest"] = c["shared"] // 2, max(1, c["longest"] // 2)
    return c


def _block(D):
    return PAGE * (3 * D // 4 + 8)


# ----------------------------------------------------------------- inputs
def _quantise(x, four):
    """Codes (0 .. 7, or 0 .. 15 where `four`) and scales of x [..., D] in fp32."""
    a = x.abs().amax(-1, keepdim=True).clamp(min=1e-5)
    Q = torch.where(four, 7.0, 3.0)
    c = torch.minimum(torch.maximum((x * (Q / a)).round(), -Q - 1), Q) + Q + 1
    return c.to(torch.int32), (a / Q).squeeze(-1)


def _rows3(c):
    """Codes [..., D] of 3 bits -> bytes [..., 3 D / 8], a little-endian bit stream."""
    w = (c.unflatten(-1, (-1, 8)) << (3 * torch.arange(8, device=c.device, dtype=torch.int32))).sum(-1, dtype=torch.int32)
    return torch.stack([w & 255, (w >> 8) & 255, w >> 16], -1).flatten(-2).to(torch.uint8)


def _rows4(c):
    """Codes [..., D] of 4 bits -> bytes [..., D / 2], low half first."""
    c = c.unflatten(-1, (-1, 2))
    return (c[..., 0] | (c[..., 1] << 4)).to(torch.uint8)


def _views(pages, D):
    """K rows [p, h, 64, rb], V bytes [p, h, 16, rb, 4] and the scales [p, h, 64] of `pages`."""
    rb = 3 * D // 8
    s = pages[..., 2 * PAGE * rb:].view(torch.float32)
    return pages[..., :PAGE * rb].unflatten(-1, (PAGE, rb)), pages[..., PAGE * rb:2 * PAGE * rb].unflatten(-1, (PAGE // 4, rb, 4)), s[..., :PAGE], s[..., PAGE:]


def _fill(pages, codes4, D, rows4, g):
    """Writes quantised random keys and values into every slot of `pages` [n, H, block]. With rows4, a few
    tokens of each page are kept at 4 bits."""
    kv, vv, ks, vs = _views(pages, D)
    n, H = pages.shape[:2]
    gain = torch.rand(2, H, 1, D, device=DEV, generator=g) * 1.5 + 0.25  # channels differ in size
    step = max(1, (1 << 26) // (H * PAGE * D))
    at = torch.arange(PAGE, device=DEV)
    for i in range(0, n, step):
        j = min(n, i + step)
        x = torch.randn(2, j - i, H, PAGE, D, device=DEV, generator=g) * gain[:, None]
        x = x.to(torch.bfloat16).float()
        # token 5 r of a page is kept in its row r
        four = (at % 5 == 0) & (at // 5 < rows4)
        c, s = _quantise(x, four[:, None])
        b = _rows3(torch.where(four[:, None], 0, c))
        b[0, ..., 0] = torch.where(four, at // 5, b[0, ..., 0]).to(torch.uint8)
        kv[i:j] = b[0]
        vv[i:j] = b[1].unflatten(2, (PAGE // 4, 4)).transpose(-1, -2)
        ks[i:j] = torch.where(four, -s[0], s[0])
        vs[i:j] = s[1]
        if rows4:
            codes4[i:j] = torch.cat([_rows4(c[0, :, :, :5 * rows4:5]), _rows4(c[1, :, :, :5 * rows4:5])], -1)


def _pool(n_pages, H, D, rows4, g, L=None):
    shape = (n_pages,) if L is None else (L, n_pages)
    pages = torch.zeros(*shape, H, _block(D), dtype=torch.uint8, device=DEV)
    codes4 = torch.zeros(*shape, H, rows4, D, dtype=torch.uint8, device=DEV) if rows4 else None
    flat = pages.view(-1, H, _block(D))
    _fill(flat, codes4.view(-1, H, rows4, D) if rows4 else None, D, rows4, g)
    return pages, codes4


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    D, H = c["D"], c["H"]
    i32 = dict(dtype=torch.int32, device=DEV)

    def ints(lo, hi, shape):
        return torch.randint(lo, hi + 1, shape, device=DEV, generator=g)

    if c["op"] == "append":
        n, Hq = c["n"], c["Hq"]
        qkv = torch.randn(n, (Hq + 2 * H) * D, device=DEV, generator=g).to(torch.bfloat16)
        k = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        v = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
        row4 = torch.full((n,), -1, **i32) if c["rows4"] else None
        if c["decode"]:  # a token for each sequence, in a page of its own
            n_pages = n
            slots = torch.randperm(n, device=DEV, generator=g) * PAGE + ints(0, PAGE - 1, (n,))
            if c["rows4"]:
                row4 = torch.where(ints(0, 7, (n,)) == 0, ints(0, c["rows4"] - 1, (n,)), -1).to(torch.int32)
        else:  # consecutive tokens of one sequence from some place on, the batch's last ones padding
            first = int(seed) % PAGE
            n_pages = (first + n + PAGE - 1) // PAGE
            t = torch.arange(n, device=DEV) + first
            slots = torch.randperm(n_pages, device=DEV, generator=g)[t // PAGE] * PAGE + t % PAGE
            slots[n - n // 50:] = -1
            if c["rows4"]:
                row4[0] = 0
        pages = torch.zeros(n_pages, H, _block(D), dtype=torch.uint8, device=DEV)
        codes4 = torch.zeros(n_pages, H, c["rows4"], D, dtype=torch.uint8, device=DEV) if c["rows4"] else None
        return dict(case=c, k=k, v=v, slots=slots.to(torch.int32), row4=row4, pages=pages, codes4=codes4)
    if c["op"] == "copy":
        pages, codes4 = _pool(c["n_pages"], H, D, c["rows4"], g, c["L"])
        at = torch.randperm(c["n_pages"], device=DEV, generator=g).to(torch.int32)
        return dict(case=c, pages=pages, codes4=codes4, src=at[:c["n"]].contiguous(), dst=at[c["n"]:2 * c["n"]].contiguous())
    if c["op"] == "beams":
        P, R, W = c["P"], c["P"] * (1 + c["C"]), c["longest"] // PAGE + 1
        lens = torch.zeros(R, **i32)
        lens[:P] = ints(1, c["longest"], (P,)).to(torch.int32)
        used = (lens[:P] + PAGE - 1) // PAGE
        n_pages = P * W + P * c["C"] + 7
        pages, codes4 = _pool(n_pages, H, D, c["rows4"], g, c["L"])
        tables = torch.full((R, W), -1, **i32)
        at = torch.randperm(n_pages, device=DEV, generator=g)[:P * W].view(P, W)
        inside = torch.arange(W, device=DEV) < used[:, None]
        tables[:P] = torch.where(inside, at, -1).to(torch.int32)
        refs = torch.zeros(n_pages, **i32)
        refs[at[inside]] = 1
        kids = torch.arange(P, R, **i32)
        return dict(case=c, pages=pages, codes4=codes4, tables=tables, lens=lens, refs=refs, kids=kids,
                    parents=((kids - P) // c["C"]).to(torch.int32), one=torch.ones(R - P, **i32))
    B, Sq, G = c["B"], c["Sq"], c["G"]
    mine = torch.full((B,), c["longest"], **i32)
    if c["ragged"]:
        mine = ints(1, c["longest"], (B,)).to(torch.int32)
    lens = mine + PAGE * c["shared"]
    if B > 4:
        lens[B // 2] = 0  # a slot of the batch without a request
        mine[B // 2] = 0
    W = max(1, (c["longest"] + PAGE - 1) // PAGE)
    inside = torch.arange(W, device=DEV) < (mine[:, None] + PAGE - 1) // PAGE
    n_pages = c["shared"] + int(inside.sum()) + 3
    at = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    tables = torch.full((B, W), -1, **i32)
    tables[inside] = at[c["shared"]:c["shared"] + int(inside.sum())]
    pages, codes4 = _pool(n_pages, H, D, c["rows4"], g)
    q = (1.5 * torch.randn(B, Sq, H * G, D, device=DEV, generator=g)).to(torch.bfloat16)
    return dict(case=c, q=q, pages=pages, codes4=codes4, tables=tables, lens=lens, shared=at[:c["shared"]].contiguous())


# --------------------------------------------------------------- the runs
def run(state):
    c = state["case"]
    if own:
        return _own(c["op"], state)
    if c["op"] == "append":
        return _append(state)
    if c["op"] == "copy":
        return _copy(state, state["src"].long(), state["dst"].long())
    if c["op"] == "beams":
        return _beams(state)
    return _attention(state)


def _own(op, s):
    import bit_quantised_gemm_b200 as B
    if op == "append":
        B.kv_append_3bit(s["k"], s["v"], s["slots"], s["pages"], row4=s["row4"], codes4=s["codes4"])
        return s["pages"], s["codes4"]
    if op == "copy":
        B.kv_pages_copy(s["pages"], s["src"], s["dst"], codes4=s["codes4"])
        return s["pages"], s["codes4"]
    if op == "beams":
        B.kv_pages_free(s["tables"], s["lens"], s["refs"], s["kids"])
        B.kv_pages_fork(s["tables"], s["lens"], s["refs"], s["parents"], s["kids"])
        slots = B.kv_pages_grow(s["pages"], s["tables"], s["lens"], s["refs"], s["kids"], s["one"], 1, codes4=s["codes4"])
        return slots, s["tables"], s["lens"], s["refs"], s["pages"], s["codes4"]
    if "workspace" not in s:
        s["workspace"] = B.kv_attention_3bit_paged_workspace(s["q"], s["pages"], s["tables"], s["shared"])
    return B.kv_attention_3bit_paged(s["q"], s["pages"], s["tables"], s["lens"], shared=s["shared"], codes4=s["codes4"],
                                     workspace=s["workspace"])


def _append(s):
    D = s["case"]["D"]
    keep = s["slots"] >= 0
    page, off = (s["slots"][keep] // PAGE).long(), (s["slots"][keep] % PAGE).long()
    x = torch.stack([s["k"][keep], s["v"][keep]]).float()
    j = torch.full_like(page, -1) if s["row4"] is None else s["row4"][keep].long()
    four = j >= 0
    c, sc = _quantise(x, four[:, None, None])
    b = _rows3(torch.where(four[:, None, None], 0, c))
    b[0, ..., 0] = torch.where(four[:, None], j[:, None], b[0, ..., 0]).to(torch.uint8)
    kv, vv, ks, vs = _views(s["pages"], D)
    kv[page, :, off] = b[0]
    vv[page, :, off // 4, :, off % 4] = b[1]
    ks[page, :, off] = torch.where(four[:, None], -sc[0], sc[0])
    vs[page, :, off] = sc[1]
    if s["codes4"] is not None:
        s["codes4"][page[four], :, j[four]] = torch.cat([_rows4(c[0, four]), _rows4(c[1, four])], -1)
    return s["pages"], s["codes4"]


def _copy(s, src, dst):
    s["pages"][:, dst] = s["pages"][:, src]
    if s["codes4"] is not None:
        s["codes4"][:, dst] = s["codes4"][:, src]
    return s["pages"], s["codes4"]


def _beams(s):
    tables, lens, refs, kids, parents = s["tables"], s["lens"], s["refs"], s["kids"].long(), s["parents"].long()
    entry = torch.arange(tables.shape[1], device=DEV)

    def count(rows, by):  # every page that the rows hold, as often as they do
        held = entry < ((lens[rows] + PAGE - 1) // PAGE)[:, None]
        page = torch.where(held, tables[rows], 0).long().flatten()
        refs.index_add_(0, page, held.flatten().to(torch.int32) * by)
        return held

    count(kids, -1)
    held = count(parents, 1)
    tables[kids] = torch.where(held, tables[parents], tables[kids])
    lens[kids] = lens[parents]
    # one more token each: a page of its own where the last one is full, or is partly filled and shared
    n = lens[kids].long()
    last = tables[kids, (n - 1) // PAGE].long()
    part = n % PAGE != 0
    before = ((last[:, None] == last) & part).tril(-1).sum(1)  # rows before this one that leave the same page
    copies = part & (refs[last] - before > 1)
    new = copies | ~part
    page = torch.where(new, torch.nonzero(refs == 0).flatten()[(new.cumsum(0) - 1).clamp(min=0)], last)
    refs.index_add_(0, last, -copies.to(torch.int32))
    refs[page[new]] = 1
    tables[kids, n // PAGE] = page.to(torch.int32)
    lens[kids] += 1
    _copy(s, last[copies], page[copies])
    return (page * PAGE + n % PAGE).to(torch.int32)[:, None], tables, lens, refs, s["pages"], s["codes4"]


def _dequant(pages, codes4, page, D):
    """K, V [n, H, 64, D] in fp32 of the pages `page` [n]."""
    kv, vv, ks, vs = _views(pages[page], D)
    out = []
    for rows, sc in ((kv, ks), (vv.transpose(-1, -2).flatten(2, 3), vs)):
        b = rows.unflatten(-1, (-1, 3)).to(torch.int32)
        w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        c = (w[..., None] >> (3 * torch.arange(8, device=DEV, dtype=torch.int32))) & 7
        out.append((c.flatten(-2) - 4).float() * sc.abs()[..., None])
    if codes4 is not None:
        four = torch.signbit(ks)[..., None]
        j = torch.where(four[..., 0], kv[..., 0], 0).long()
        b = codes4[page].gather(2, j[..., None].expand(-1, -1, -1, D)).to(torch.int32)
        c = torch.stack([b & 15, b >> 4], -1).flatten(-2) - 8
        out = [torch.where(four, c[..., i * D:(i + 1) * D].float() * sc.abs()[..., None], x)
               for i, (x, sc) in enumerate(zip(out, (ks, vs)))]
    return out


def _attention(s):
    q, lens, shared, tables = s["q"].float(), s["lens"].long(), s["shared"].long(), s["tables"].long()
    B, Sq, Hq, D = q.shape
    H = s["case"]["H"]
    W, T0 = tables.shape[1], PAGE * len(shared)
    q = q.unflatten(2, (H, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3) / math.sqrt(D)  # [B, H, G Sq, D]
    k, v = _dequant(s["pages"], s["codes4"], tables.clamp(min=0).flatten(), D)
    k, v = (x.unflatten(0, (B, W)).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [B, H, W 64, D]
    score = q @ k.transpose(-1, -2)
    if T0:
        k0, v0 = (x.transpose(0, 1).flatten(1, 2) for x in _dequant(s["pages"], s["codes4"], shared, D))  # [H, T0, D]
        first = (q.transpose(0, 1).flatten(1, 2) @ k0.transpose(-1, -2)).unflatten(1, (B, -1)).transpose(0, 1)
        score = torch.cat([first, score], -1)
    sees = lens[:, None] - Sq + 1 + torch.arange(Sq, device=DEV)  # tokens that each query sees
    sees = sees.repeat(1, Hq // H)[:, None, :, None]
    mask = torch.arange(T0 + W * PAGE, device=DEV) < sees
    score = torch.where(mask, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    # pages behind the last token hold what they hold: their values take no part
    seen = (torch.arange(W * PAGE, device=DEV) + T0 < lens[:, None])[:, None, :, None]
    o = p[..., T0:] @ torch.where(seen, v, 0.0)
    if T0:
        o = o + (p[..., :T0].transpose(0, 1).flatten(1, 2) @ v0).unflatten(1, (B, -1)).transpose(0, 1)
    o = torch.where(total > 0, o / total, 0.0)
    return o.unflatten(2, (-1, Sq)).permute(0, 3, 1, 2, 4).flatten(2, 3).to(torch.bfloat16)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    D, H = c["D"], c["H"]
    token = H * (3 * D // 4 + 8)  # bytes of a cached token
    if c["op"] == "append":
        n = c["n"] if c["decode"] else c["n"] - c["n"] // 50
        return dict(bytes=n * (4 * H * D + token + 4), flops=10 * n * H * D)
    page = PAGE * token + c["rows4"] * H * D
    if c["op"] == "copy":
        return dict(bytes=2 * c["n"] * c["L"] * page + 8 * c["n"], flops=0)
    if c["op"] == "beams":
        n = c["P"] * c["C"]
        held = (c["longest"] / 2 + PAGE / 2) / PAGE  # pages of a sequence, on average
        return dict(bytes=int(2 * n * c["L"] * page * (1 - 1 / PAGE) + n * held * 4 * 6 + 4 * 2 * n), flops=0)
    B, Hq = c["B"], H * c["G"]
    live = B - 1 if B > 4 else B
    mine = live * ((1 + c["longest"]) / 2 if c["ragged"] else c["longest"])
    return dict(bytes=int((mine + PAGE * c["shared"]) * token + B * c["Sq"] * Hq * D * 4),
                flops=int(4 * D * Hq * c["Sq"] * (mine + live * PAGE * c["shared"])))


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """Attention in 64 bits, sequence by sequence from the definition. What the
    other operators write is whole numbers, decided in 32 bits."""
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    q, D, H, G, Sq = s["q"].double(), case["D"], case["H"], case["G"], case["Sq"]
    rb = 3 * D // 8
    three = torch.tensor([1.0, 2.0, 4.0], dtype=torch.float64, device=DEV)
    eight = torch.arange(8, device=DEV, dtype=torch.uint8)

    def rows(ids, which):  # [tokens, H, D] of the tokens in the pages `ids`
        raw = s["pages"][ids]
        code = raw[..., which * PAGE * rb:(which + 1) * PAGE * rb]
        if which:
            code = code.reshape(len(ids), H, PAGE // 4, rb, 4).movedim(-1, -2)
        code = code.reshape(len(ids), H, PAGE, rb)
        bits = ((code[..., None] >> eight) & 1).reshape(len(ids), H, PAGE, D, 3)
        value = bits.double() @ three - 4
        scale = raw[..., 2 * PAGE * rb:].contiguous().view(torch.float32).view(len(ids), H, 2, PAGE)
        if case["rows4"]:
            four = scale[:, :, 0] < 0
            p, h, t = torch.nonzero(four, as_tuple=True)
            j = raw[p, h, t * rb].long()
            b = s["codes4"][ids][p, h, j, which * D // 2:(which + 1) * D // 2].double()
            value[p, h, t, 0::2] = torch.remainder(b, 16) - 8
            value[p, h, t, 1::2] = torch.floor(b / 16) - 8
        value = value * scale[:, :, which].double().abs()[..., None]
        return value.transpose(1, 2).reshape(-1, H, D)

    front = [rows(s["shared"].long(), i) for i in (0, 1)]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        own_pages = max(0, -(-(n - PAGE * case["shared"]) // PAGE))
        k, v = (torch.cat([f, rows(s["tables"][b, :own_pages].long(), i)])[:n] for i, f in enumerate(front))
        for i in range(Sq):
            m = n - Sq + 1 + i
            if m > 0:
                z = torch.einsum("hgd,thd->hgt", q[b, i].view(H, G, D), k[:m]) / D ** 0.5
                z = torch.softmax(z, -1)
                out[b, i] = torch.einsum("hgt,thd->hgd", z, v[:m]).reshape(H * G, D)
    return out
