"""The paged 8-bit key/value cache on the GPU: plan, append and attention
against plain implementations in 64 bits.

Tolerances, derived from the arithmetic (o: output of a row, t_j = s_j + log2 b_j
its logits to base 2 with the value scale b_j taken in, m their maximum,
w_j = 2^(t_j - m) / l the weights with l = sum_j 2^(t_j - m) / b_j):
  - the output is rounded once to bf16: 2^-8 |o|, and 2^-134 below its normal range;
  - a weight held as e4m3 hi + lo is off by at most 2^-4 * 2^-4 = 2^-8 of itself, or
    half of lo's smallest step, 2^-10, on a scale where the largest weight is at least 2^4:
    2^-14 of the largest (a tile's weights may be held below a maximum that is
    itself allowed to be 2^4 too small): sum_j (2^-8 w_j + 2^-14 / l) |c_j|;
  - q held as hi + lo is off by at most 2^-10 on a scale where its largest is at
    least 224, that is max|q| * 2^-17 an element; the fp32 sums of d products, taken
    in any order and truncated, are off by at most d 2^-23 sum |q c|; ex2 and the
    fused steps by 2^-21 + |t| 2^-22.  A logit's error ds (in powers of two)
    moves the output by at most ln 2 * 2 max_j ds_j * sum_j w_j |c_j| and the lse by
    ln 2 max_j ds_j;
  - sums of L weights in fp32, in any order: L 2^-24 relative, doubled."""
import ctypes
import math
import os

import pytest
import torch

from hybrid_linear_attention_conv_gb300 import gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN_CODE = 0x7F


@pytest.fixture(scope="module", autouse=True)
def _built():
    from hybrid_linear_attention_conv_gb300 import build
    build.build()
    gdn.load()
    assert torch.cuda.is_available()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def plan_ref(lens, add, held, free, count, table, page, rows):
    """The plan in plain Python; (table, lens, held, count, start, slots, status)."""
    B, width = len(lens), len(table[0]) if table else 0
    table = [list(r) for r in table]
    status, need, total = 0, 0, 0
    want = []
    for b in range(B):
        want.append(max(held[b], -(-(lens[b] + add[b]) // page)))
        if lens[b] < 0 or add[b] < 0 or held[b] < 0 or held[b] > width:
            status |= 8
            continue
        if want[b] > width:
            status |= 2
        need += want[b] - held[b]
        total += add[b]
    if count < 0 or count > len(free):
        status |= 8
    if need > count:
        status |= 1
    if total > rows:
        status |= 4
    if status:
        return table, lens, held, count, [0] * (B + 1), [-1] * rows, status
    start, slots = [0], []
    top = count
    for b in range(B):
        for j in range(held[b], want[b]):
            top -= 1
            table[b][j] = free[top]
        slots += [table[b][p // page] * page + p % page for p in range(lens[b], lens[b] + add[b])]
        start.append(start[-1] + add[b])
    return table, [a + b for a, b in zip(lens, add)], want, top, start, slots + [-1] * (rows - len(slots)), 0


def run_plan(lens, add, held, free, count, table, page, rows):
    t = i32(table) if table else torch.empty((0, 1), dtype=torch.int32, device=DEV)
    got = gdn.kv_plan(i32(lens), i32(add), i32(held), i32(free), i32([count]), t, page, rows)
    torch.cuda.synchronize()
    lens_o, held_o, count_o, start, slots, status = (x.tolist() for x in got)
    return t.tolist(), lens_o, held_o, count_o[0], start, slots, status[0]


def plan_case(seed, B, page, ctx_hi, new_hi, extra_rows=3):
    import random
    r = random.Random(seed)
    lens = [r.randint(0, ctx_hi) for _ in range(B)]
    add = [r.choice([0, 1, r.randint(0, new_hi)]) for _ in range(B)]
    held = [-(-x // page) + r.choice([0, 0, 1, 2]) for x in lens]  # some hold more than their length needs
    width = max([-(-(x + a) // page) for x, a in zip(lens, add)] + held + [1])
    ids = list(range(sum(held) + sum(add) // page + B + 5))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:]
    return lens, add, held, free, len(free) - 2, table, page, sum(add) + extra_rows


@pytest.mark.parametrize("seed,B,page,ctx_hi,new_hi", [
    (0, 1, 32, 0, 1), (1, 1, 64, 100, 5000), (2, 3, 128, 500, 300), (3, 64, 64, 1000, 1), (4, 511, 32, 200, 70),
    (5, 513, 64, 2000, 40), (6, 1500, 128, 300, 130), (7, 12288, 32, 60, 2), (8, 17, 32, 31, 33)])
def test_plan(seed, B, page, ctx_hi, new_hi):
    c = plan_case(seed, B, page, ctx_hi, new_hi)
    assert run_plan(*c) == tuple(plan_ref(*c))


def test_plan_exact_fits_and_refusals():
    lens, add, held, free, count, table, page, rows = plan_case(11, 40, 64, 400, 200, extra_rows=0)
    need = sum(max(0, -(-(x + a) // page) - h) for x, a, h in zip(lens, add, held))
    assert need > 2 and need <= count
    for status, kw in ((0, dict(count=need)), (1, dict(count=need - 1)), (4, dict(rows=rows - 1)), (0, dict(rows=rows)),
                       (8, dict(count=len(free) + 1)), (8 | 1, dict(count=-1))):
        c = dict(lens=lens, add=add, held=held, free=free, count=count, table=table, page=page, rows=rows) | kw
        got, want = run_plan(**c), plan_ref(**c)
        assert got == tuple(want) and got[-1] == status
    for name, bad in (("lens", -1), ("add", -2), ("held", -1), ("held", len(table[0]) + 1)):
        c = dict(lens=list(lens), add=list(add), held=list(held), free=free, count=count, table=table, page=page, rows=rows)
        c[name][7] = bad
        got = run_plan(**c)
        assert got[-1] & 8 and got[0] == table and got[4] == [0] * 41 and got[5] == [-1] * rows
    grow = list(add)
    grow[5] = len(table[0]) * page - lens[5] + 1  # one token more than its table row holds
    got = run_plan(lens, grow, held, free, count, table, page, rows + grow[5])
    assert got[-1] & 2 and got[0] == table
    with pytest.raises(gdn.GdnError):
        gdn.kv_plan_check(i32([2]))
    gdn.kv_plan_check(i32([0]))


def test_plan_of_no_requests():
    got = run_plan([], [], [], [3, 4], 2, [], 32, 4)
    assert got[1:] == ([], [], 2, [0], [-1] * 4, 0)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def nearest_e4m3(y):
    _, e = torch.frexp(y)
    step = torch.exp2((e.double() - 4.0).clamp(min=-9.0))
    return torch.round(y / step) * step


def append_ref(k, v, slots, kc, vc, ks, vs, page, rows=None):
    """In 64 bits, on copies: codes' values and scales of both caches."""
    runs = {}
    for t, s in enumerate(slots):
        if 0 <= s < kc.shape[0] * page:
            runs.setdefault(s // page, []).append((s % page, t))
    out = []
    for x, c, sc in ((k, kc, ks), (v, vc, vs)):
        x, c, sc = x.double().cpu(), c.double().cpu(), sc.double().cpu().clone()
        for pg, members in runs.items():
            first, n = members[0][0], len(members)
            src = [rows[t] if rows is not None else t for _, t in members]
            block = torch.stack([x[s] if 0 <= s < x.shape[0] else torch.full_like(x[0], math.nan) for s in src]).transpose(0, 1)
            fin = torch.isfinite(block)
            block = torch.where(fin, block, 0.0)
            m, e = torch.frexp(block.abs().amax((1, 2)) / 448.0)
            now = torch.exp2((e - (m == 0.5).int()).double().clamp(-100, 120))
            now = torch.where(block.abs().amax((1, 2)) == 0, 2.0 ** -100, now)
            for h in range(x.shape[1]):
                old = sc[pg, h].item() if first else 0.0
                if first and not (0 < old < math.inf):
                    sc[pg, h] = math.nan
                    c[pg, h, first:first + n] = nearest_e4m3(block[h] / now[h])
                    continue
                s = max(old, now[h].item())
                if first and s > old:
                    c[pg, h, :first] = nearest_e4m3(c[pg, h, :first] * (old / s))
                c[pg, h, first:first + n] = nearest_e4m3(block[h] / s)
                sc[pg, h] = s if fin[h].all() else math.nan
        out += [c, sc]
    return out


def new_cache(pages, Hkv, page, d, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = [(torch.randn((pages, Hkv, page, d), generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2)]
    s = [torch.exp2(torch.randint(-9, -5, (pages, Hkv), generator=g, device=DEV).float()) for _ in range(2)]
    return c[0], c[1], s[0], s[1]


def check_append(k, v, slots, cache, page, rows=None):
    want = append_ref(k, v, slots, *cache, page, rows)
    gdn.kv_append(k, v, torch.tensor(slots, dtype=torch.int64, device=DEV), *cache, rows=None if rows is None else i32(rows))
    torch.cuda.synchronize()
    kc, vc, ks, vs = cache
    for got, ref in ((ks, want[1]), (vs, want[3]), (kc, want[0]), (vc, want[2])):
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))  # every code and scale, exactly


def rows_of(T, Hkv, d, seed, spread=3.0):
    """k and v as slices of wider rows, tokens of very different sizes among them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, 3 * Hkv * d), generator=g, device=DEV) * torch.exp2(spread * torch.randn((T, 1), generator=g, device=DEV))
    x = x.to(torch.bfloat16)
    return x[:, Hkv * d:2 * Hkv * d].view(T, Hkv, d), x[:, 2 * Hkv * d:].view(T, Hkv, d)


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("Hkv,lens", [
    (1, [(0, 1)]), (2, [(0, 300), (5, 1), (31, 2), (32, 4), (63, 5), (127, 130), (64, 64)]),
    (4, [(17, 1)] * 9 + [(0, 1)] * 9), (3, [(1, 33), (2, 6), (3, 7), (100, 8), (90, 40), (0, 1500)])])
def test_append(page, d, Hkv, lens):
    slots, at = [], 0
    order = torch.randperm(400, generator=torch.Generator().manual_seed(page + d)).tolist()
    for ctx, n in lens:
        table = order[at:at + -(-(ctx + n) // page)]
        at += len(table)
        slots += [table[p // page] * page + p % page for p in range(ctx, ctx + n)]
    k, v = rows_of(len(slots), Hkv, d, seed=d + len(slots))
    check_append(k, v, slots, new_cache(400, Hkv, page, d), page)


def test_append_token_by_token_moves_older_codes_by_powers_of_two():
    page, d, Hkv = 64, 128, 2
    cache = new_cache(3, Hkv, page, d)
    k, v = rows_of(100, Hkv, d, seed=5, spread=4.0)
    for t in range(100):
        s = 128 + t if t < 64 else t - 64
        check_append(k[t:t + 1], v[t:t + 1], [s], cache, page)


def test_append_skips_and_gathers():
    page, d, Hkv = 32, 128, 4
    k, v = rows_of(50, Hkv, d, seed=6)
    slots = [-1, 64, 65, -1, 66, 67, 10 ** 12, 5 * 32, -(10 ** 12), 32 * 20, 31, 7 * 32]
    rows = [0, 49, 3, 3, 3, 17, 0, 8, 9, 1, 2, 44]
    # 64.. is two runs in one page: the second one is a call of its own below
    check_append(k, v, slots[:4] + [-1, -1] + slots[6:], new_cache(20, Hkv, page, d), page, rows)
    # a source row that does not exist makes the block NaN, and nothing else is touched
    check_append(k, v, [32, 33, 96], new_cache(20, Hkv, page, d), page, [4, 50, 3])
    check_append(k, v, [32, 33, 96], new_cache(20, Hkv, page, d), page, [4, -1, 3])


@pytest.mark.parametrize("n", [2, 30])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_append_values_that_are_not_finite(bad, n):
    page, d, Hkv = 32, 256, 2
    cache = new_cache(4, Hkv, page, d)
    k, v = rows_of(64, Hkv, d, seed=7)
    k, v = k.clone(), v.clone()
    k[1, 1, 200] = bad
    check_append(k[:n], v[:n], list(range(32, 32 + n)), cache, page)      # begins the block
    assert torch.isnan(cache[2][1, 1]) and not torch.isnan(cache[2][1, 0])
    check_append(k[40:41], v[40:41], [32 + n], cache, page)               # the block stays NaN
    assert torch.isnan(cache[2][1, 1])
    check_append(k[41:43], v[41:43], [32, 33], cache, page)               # begun again, it is well
    assert not torch.isnan(cache[2][1, 1])


def test_append_zeros_and_extremes():
    page, d, Hkv = 32, 128, 1
    k = torch.zeros((6, Hkv, d), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[1], k[2], k[3] = 3.3e38, 1e-38, 448.0
    v[1], v[2], v[3] = -3.3e38, 9e-41, 449.0
    for n, slot in ((1, 0), (6, 32), (1, 64)):
        check_append(k[:n], v[:n], list(range(slot, slot + n)), new_cache(4, Hkv, page, d), page)
    check_append(k[2:3], v[2:3], [96], new_cache(4, Hkv, page, d), page)
    check_append(k[3:4], v[3:4], [96], new_cache(4, Hkv, page, d), page)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Step:
    """Requests over a cache whose every byte that a request does not own, or that lies
    past its length, is NaN: codes and scales."""

    def __init__(self, lens, new, Hq, Hkv, d, page, seed, sharp=1.0, v_exp=(-9, -5), spare_width=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.page, self.L, self.n = Hq, Hkv, d, page, lens, new
        held = [-(-x // page) for x in lens]
        self.pages = sum(held) + 3
        self.cache = list(new_cache(self.pages, Hkv, page, d, seed))
        self.cache[3] = torch.exp2(torch.randint(v_exp[0], v_exp[1], (self.pages, Hkv), generator=g, device=DEV).float())
        order = torch.randperm(self.pages, generator=g, device=DEV).tolist()
        width = max(held + [1]) + spare_width
        table, at = [], 0
        owned = torch.zeros((self.pages, page), dtype=torch.bool, device=DEV)
        for h, x in zip(held, lens):
            mine = order[at:at + h]
            at += h
            for j, pg in enumerate(mine):
                owned[pg, :min(page, x - j * page)] = True
            table.append(mine + [-1] * (width - h))
        self.owned = owned
        for c in self.cache[:2]:
            c.view(torch.uint8).masked_fill_(~owned[:, None, :, None], NAN_CODE)
        for s in self.cache[2:]:
            s.masked_fill_(~owned.any(1)[:, None], math.nan)
        self.table = i32(table)
        starts = [0]
        for x in new:
            starts.append(starts[-1] + x)
        self.start_list, self.T = starts, starts[-1]
        self.start, self.lens = i32(starts), i32(lens)
        row = torch.randn((max(self.T, 1), (Hq + 3) * d), generator=g, device=DEV) * sharp
        self.q = row.to(torch.bfloat16)[:self.T, 2 * d:(Hq + 2) * d].view(self.T, Hq, d)
        self.tree = None

    def with_trees(self, seed=0):
        import random
        r = random.Random(seed)
        words = []
        for n in self.n:
            mask = []
            for i in range(n):
                mask.append((mask[r.randint(max(0, i - 5), i - 1)] if i and r.random() < 0.95 else 0) | (1 << i if i < 64 else 0))
            words += mask
        self.tree = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=DEV)
        return self

    def run(self, scale=None, workspace=None, tiles=False, pad=2):
        """pad: rows of q past the requests' own.  The rows a request and the table's width, which
        bounds the contexts, pick the kernel: tiles adds enough of both for the one of 128 rows at a
        time; without it few rows go to the one of eight."""
        table, B = self.table, len(self.L)
        if tiles:
            pad = 9 * B
            more = ((1 << 22) // (B * self.Hkv) + 8192) // self.page
            table = torch.cat([table, table.new_full((B, more), -1)], 1)
        out = torch.full((self.T + pad, self.Hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV)  # rows that no request has stay
        lse = torch.full((self.T + pad, self.Hq), 7.0, device=DEV)
        q = torch.cat([self.q, self.q.new_zeros((pad, self.Hq, self.d))])
        tree = None if self.tree is None else torch.cat([self.tree, self.tree.new_zeros(pad)])
        gdn.kv_attention(q, *self.cache, table, self.start, self.lens, scale=scale, tree=tree, out=out, lse=lse, workspace=workspace)
        torch.cuda.synchronize()
        assert (out[self.T:] == 7.0).all() and (lse[self.T:] == 7.0).all()
        return out[:self.T], lse[:self.T]

    def check(self, scale=None, got=None, tiles=False):
        out, lse = got or self.run(scale, tiles=tiles)
        scale = self.d ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        kc, vc = (c.view(torch.uint8) for c in self.cache[:2])
        for b, (L, n) in enumerate(zip(self.L, self.n)):
            if n == 0:
                continue
            t0 = self.start_list[b]
            pages = self.table[b, :-(-L // self.page)].long()
            j = torch.arange(L, device=DEV)[None]
            base = L - n
            i = torch.arange(n, device=DEV)[:, None]
            if self.tree is None:
                seen = j <= base + i
            else:
                bit = (self.tree[t0:t0 + n, None] >> (j - base).clamp(0, 63)) & 1
                seen = (j < base) | ((bit == 1) & (j - base < 64))
            for h in range(self.Hkv):
                def of(c, s):
                    codes = c[pages, h].view(torch.float8_e4m3fn).double().reshape(-1, self.d)[:L]
                    return codes, s[pages, h].double().repeat_interleave(self.page)[:L]
                K, a = of(kc, self.cache[2])
                V, w = of(vc, self.cache[3])
                q = self.q[t0:t0 + n, h * G:(h + 1) * G].double().transpose(0, 1)  # [G, n, d]
                raw = q @ K.T * a                                          # natural logits / scale
                t = (raw * scale * math.log2(math.e) + w.log2()).masked_fill(~seen, -math.inf)
                m = t.amax(-1, keepdim=True).clamp(min=-1e300) if L else torch.zeros((G, n, 1), device=DEV, dtype=torch.float64)
                p = torch.exp2(t - m)
                l = (p / w).sum(-1, keepdim=True)
                some = l > 0
                o = torch.where(some, (p @ V) / l, 0.0)
                z = torch.where(some, (m + l.log2()) * math.log(2), -math.inf)[..., 0]
                ds = scale * math.log2(math.e) * (a * (q.abs().amax(-1, keepdim=True) * 2.0 ** -17 * K.abs().sum(-1)
                                                       + self.d * 2.0 ** -23 * (q.abs() @ K.abs().T)))
                ds = ds + 2.0 ** -21 + t.abs().masked_fill(~seen, 0) * 2.0 ** -22
                ds = ds.masked_fill(~seen, 0).amax(-1, keepdim=True) if L else ds.sum(-1, keepdim=True)
                size = torch.where(some, (p @ V.abs()) / l, 0.0)
                bound = (2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * math.log(2) * ds + L * 2.0 ** -23) * size
                         + torch.where(some, 2.0 ** -14 * (seen.double() @ V.abs()) / l, 0.0) + 1e-38)
                got_o = out[t0:t0 + n, h * G:(h + 1) * G].double().transpose(0, 1)
                got_z = lse[t0:t0 + n, h * G:(h + 1) * G].double().transpose(0, 1)
                assert torch.isfinite(got_o).all(), (b, h)
                assert ((got_o - o).abs() <= bound).all(), (b, h, float(((got_o - o).abs() / bound).max()))
                assert torch.equal(torch.isinf(got_z), torch.isinf(z))
                fine = torch.isfinite(z)
                err = (got_z - z).abs()[fine]
                lim = (math.log(2) * ds[..., 0] + L * 2.0 ** -23 + z.abs() * 2.0 ** -22 + 2.0 ** -20)[fine]
                assert (err <= lim).all(), (b, h, float((err / lim).max()))
        return out, lse


SHAPES = [(24, 4, 256), (8, 8, 128), (16, 2, 128), (3, 1, 256), (32, 8, 128), (10, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("tiles", [False, True])
def test_attention_one_token(Hq, Hkv, d, page, tiles):
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1025]
    Step(lens, [1] * len(lens), Hq, Hkv, d, page, seed=page + d).check(tiles=tiles)


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("tiles", [False, True])
def test_attention_prompts_and_single_tokens(Hq, Hkv, d, tiles):
    Step([40, 7, 300, 129, 1, 513, 64, 0], [40, 1, 130, 0, 1, 5, 64, 0], Hq, Hkv, d, 64, seed=d).check(tiles=tiles)


@pytest.mark.parametrize("Hq,Hkv,d", [(24, 4, 256), (8, 8, 128), (16, 1, 128)])
@pytest.mark.parametrize("n", [1, 2, 7, 32, 63, 64])
@pytest.mark.parametrize("tiles", [False, True])
def test_attention_trees(Hq, Hkv, d, n, tiles):
    Step([n, n + 1, n + 31, n + 700], [n] * 4, Hq, Hkv, d, 32, seed=n).with_trees(n).check(tiles=tiles)


@pytest.mark.parametrize("tiles", [False, True])
def test_attention_tree_of_more_nodes_than_bits(tiles):
    Step([70, 200], [70, 66], 8, 2, 128, 64, seed=3).with_trees().check(tiles=tiles)


@pytest.mark.parametrize("tiles", [False, True])
def test_attention_rows_that_see_nothing(tiles):
    """More queries than tokens: the first of them see none."""
    s = Step([3, 0, 40, 0], [5, 2, 41, 1], 8, 2, 128, 32, seed=4)
    out, lse = s.check(tiles=tiles)
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and (out[5:7] == 0).all()
    s = Step([30, 64], [30, 3], 6, 1, 256, 32, seed=5).with_trees()
    s.tree[:] = 0
    out, lse = s.check(tiles=tiles)
    assert (out[:30] == 0).all() and torch.isneginf(lse[:30]).all() and torch.isfinite(lse[30:]).all()


@pytest.mark.parametrize("sharp,v_exp", [(8.0, (-9, -5)), (0.01, (-9, -5)), (1.0, (-60, 40)), (30.0, (-20, 20))])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_peaked_flat_and_mixed_scales(sharp, v_exp, new):
    for tiles in (False, True):
        Step([2000, 555], [new, min(new, 20)], 12, 2, 128, 64, seed=8, sharp=sharp, v_exp=v_exp).check(tiles=tiles)
        Step([700], [new], 6, 1, 256, 128, seed=9, sharp=sharp, v_exp=v_exp).check(tiles=tiles)


def test_attention_growing_maximum():
    """Logits that rise along the context: every tile brings a new maximum."""
    for new, tiles in ((1, False), (1, True), (140, False), (140, True)):
        s = Step([3000], [new], 8, 1, 128, 64, seed=10)
        ramp = torch.linspace(0, 400, 64 * 48, device=DEV)[:s.page * s.table.shape[1]]
        s.q = torch.zeros_like(s.q)
        s.q[..., 0] = 1.0
        for j in range(-(-3000 // 64)):
            pg = int(s.table[0, j])
            s.cache[0][pg, 0, :, 0] = ramp[j * 64:(j + 1) * 64].to(torch.float8_e4m3fn)
        s.cache[0].view(torch.uint8).masked_fill_(~s.owned[:, None, :, None], NAN_CODE)
        s.cache[2].fill_(1.0)
        s.check(scale=0.5, tiles=tiles)


@pytest.mark.parametrize("Hq,Hkv,d,new", [(24, 4, 256, 1), (24, 4, 256, 32), (8, 2, 128, 1), (32, 8, 128, 700)])
@pytest.mark.parametrize("tiles", [False, True])
def test_attention_long_context_and_same_bits(Hq, Hkv, d, new, tiles):
    s = Step([20011], [new], Hq, Hkv, d, 64, seed=12)
    ws = torch.zeros(gdn.kv_attention_workspace_bytes(Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    first = s.check(got=s.run(workspace=ws, tiles=tiles))
    for _ in range(3):
        again = s.run(workspace=ws, tiles=tiles)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
    assert gdn.kv_attention_status(ws) == 0


def test_attention_many_requests():
    lens = [(37 * i) % 700 for i in range(300)]
    for tiles in (False, True):
        Step(lens, [1 if x else 0 for x in lens], 8, 2, 128, 32, seed=13).check(tiles=tiles)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("tiles", [False, True])
def test_attention_not_a_number_stays_in_its_rows(new, tiles):
    s = Step([200, 90], [new, 1], 16, 2, 128, 64, seed=14)
    clean = s.run(tiles=tiles)
    # a query
    q = s.q.clone()
    s.q[new // 2, 3, 5] = math.inf
    out, lse = s.run(tiles=tiles)
    rows = torch.zeros(out.shape[:2], dtype=torch.bool, device=DEV)
    rows[new // 2, 3] = True
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])
    s.q = q
    # a block: page 3 of the first request, tokens 192 ..., head 1
    for which in (2, 3):
        keep = s.cache[which].clone()
        s.cache[which][int(s.table[0, 3]), 1] = math.nan
        out, lse = s.run(tiles=tiles)
        rows[:] = False
        for i in range(new):
            if 200 - new + i >= 192:
                rows[i, 8:16] = True
        assert rows.any() and torch.isnan(out[rows]).all()
        assert torch.equal(out[~rows], clean[0][~rows]) and torch.equal(lse[~rows], clean[1][~rows])
        s.cache[which] = keep
    # a table entry outside the cache (kernels check it: the page reads as NaN)
    for entry in (-1, s.pages, 2 ** 31 - 1, -2 ** 31):
        keep = s.table.clone()
        s.table[0, 3] = entry
        out, lse = s.run(tiles=tiles)
        rows[:] = False
        for i in range(new):
            if 200 - new + i >= 192:
                rows[i] = True
        assert torch.isnan(out[rows]).all() and torch.equal(out[~rows], clean[0][~rows])
        s.table = keep


def test_attention_length_past_the_table_is_cut():
    """lens beyond the table's width: what the table has counts, and nothing else is read."""
    s = Step([64, 64], [1, 1], 8, 2, 128, 32, seed=15, spare_width=0)
    for pad in (0, 6000):  # of so many rows the kernel of 128 at a time takes any table's
        s.lens = i32([64, 64])
        ref = s.run(pad=pad)
        s.lens = i32([64, 10 ** 9])
        out = s.run(pad=pad)
        assert torch.equal(out[0][0], ref[0][0])


def test_attention_on_another_stream_and_in_a_graph():
    s = Step([900, 33], [1, 1], 24, 4, 256, 64, seed=16)
    ref = s.run()
    side = torch.cuda.Stream()
    ws = torch.zeros(gdn.kv_attention_workspace_bytes(24, 4, 256), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(s.q)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gdn.kv_attention(s.q, *s.cache, s.table, s.start, s.lens, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, ref[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.kv_attention(s.q, *s.cache, s.table, s.start, s.lens, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0])
    # the same graph after the lengths have moved on
    s.lens.copy_(i32([800, 20]))
    s.L = [800, 20]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, s.run()[0])


@pytest.mark.parametrize("new,tiles", [(1, False), (100, True)])
def test_attention_timeout_is_readable_and_recovers(new, tiles):
    """A wait limit of 0 makes the waits for copies just requested give up at their first
    empty probe (over a context whose copies cannot all have landed by the time they are
    waited for); the kernel still lets them land before it ends."""
    s = Step([200000], [new], 24, 4, 256, 64, seed=17)
    ws = torch.zeros(gdn.kv_attention_workspace_bytes(24, 4, 256), dtype=torch.uint8, device=DEV)
    prev = gdn.set_wait_limit_ns(0)
    try:
        s.run(workspace=ws, tiles=tiles)
        assert gdn.kv_attention_status(ws) != 0
    finally:
        gdn.set_wait_limit_ns(prev)
    ws.zero_()
    s.check(got=s.run(workspace=ws, tiles=tiles))
    assert gdn.kv_attention_status(ws) == 0


def test_cache_past_32_bits():
    """A cache of more than 2^32 bytes: the last pages are appended to and attended over."""
    page, Hkv, d = 64, 4, 256
    pages = (1 << 32) // (page * Hkv * d) + 9
    kc, vc = (torch.empty((pages, Hkv, page, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), math.nan, device=DEV) for _ in range(2))
    T = 150
    k, v = rows_of(T, Hkv, d, seed=18, spread=0.5)
    table = [pages - 1, pages - 5, pages - 3]
    slots = [table[p // page] * page + p % page for p in range(T)]
    for c in (kc, vc):
        c.view(torch.uint8)[pages - 6:] = NAN_CODE
    gdn.kv_append(k, v, torch.tensor(slots, dtype=torch.int64, device=DEV), kc, vc, ks, vs)
    small = [torch.empty((3, Hkv, page, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    small_s = [torch.full((3, Hkv), math.nan, device=DEV) for _ in range(2)]
    gdn.kv_append(k, v, torch.arange(T, device=DEV), *small, *small_s)
    q = torch.randn((T, 24, d), device=DEV).to(torch.bfloat16)
    for n in (1, T):
        big = gdn.kv_attention(q[:n], kc, vc, ks, vs, i32([table]), i32([0, n]), i32([T]))
        ref = gdn.kv_attention(q[:n], *small, *small_s, i32([[0, 1, 2]]), i32([0, n]), i32([T]))
        assert torch.isfinite(big.float()).all() and torch.equal(big, ref)
