"""Writing, reading and moving pages of the key-value cache (GPU), against
plain host forms; everything here is exact."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import int4_weight_quantized_amd as pkg
    return pkg


INV127 = torch.tensor(1.0 / 127.0, dtype=torch.float32)


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32
                  if t.dtype == torch.float32 else t.dtype)


def random_pool(w4, layers, pages, heads, ps, D, kv, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (layers, pages, heads, ps, D)
    if kv == "bf16":
        return w4.KVCache(*(torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2)))
    return w4.KVCache(*(torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).cuda()
                        for _ in range(2)),
                      *(torch.rand(shape[:4], generator=g).cuda() for _ in range(2)))


def arrays(c):
    return [t for t in (c.k, c.v, c.k_scale, c.v_scale) if t is not None]


# ------------------------------------------------------------------- append
def plain_append(c, layer, k, v, table, start, cu):
    """The host form, in place on copies of the arrays: fp32 product and division."""
    pools = [t.clone().cpu() for t in arrays(c)]
    table, start = table.tolist(), start.tolist()
    rows = [(b, p, r) for b in range(len(start))
            for p, r in enumerate(range(cu[b], cu[b + 1]))]
    for which, x in ((0, k.cpu()), (1, v.cpu())):
        for b, p, r in rows:
            if start[b] < 0:
                continue
            j = (start[b] + p) // c.page_size
            page = table[b][j] if j < len(table[b]) else -1
            if not 0 <= page < c.pages:
                continue
            slot = (start[b] + p) % c.page_size
            if c.int8:
                f = x[r].float()
                s = f.abs().amax(-1) * INV127
                q = torch.where(s[:, None] > 0, torch.round(f / s[:, None]).clamp(-128, 127), 0.0)
                pools[which][layer, page, :, slot] = q.to(torch.int8)
                pools[2 + which][layer, page, :, slot] = s
            else:
                pools[which][layer, page, :, slot] = x[r].bfloat16()
    return pools


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads,ps,D", [(2, 16, 128), (3, 32, 64), (1, 16, 256), (5, 16, 80),
                                        (2, 128, 16), (7, 16, 240)])
def test_append(w4, heads, ps, D, dt, kv):
    new = [3, 0, 1, 17, 40, 2, 5]
    start = [0, 5, 15, 16, 30, -1, 200]
    cu = [sum(new[:i]) for i in range(len(new) + 1)]
    c = random_pool(w4, 2, 40, heads, ps, D, kv, 1)
    W = 6
    order = random.Random(2).sample(range(40), 40)
    table = [[order[b * 5 + j] if j < 5 else -1 for j in range(W)] for b in range(7)]
    table[3][1] = 40
    table[4][2] = -9
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((cu[-1], heads, D), generator=g).to(dt).cuda() for _ in range(2))
    k[2] = 0.0  # an all-zero vector: scale 0, codes 0
    v[3, :, 0] = 1e-30
    want = plain_append(c, 1, k, v, ints(table), ints(start), cu)
    w4.kv_append(c, 1, k, v, ints(table), ints(start), ints(cu))
    for a, b in zip(arrays(c), want):
        assert torch.equal(bits(a.cpu()), bits(b))
    # read back: the values that the cache holds, zeros where there is no page
    gk, gv = w4.kv_gather(c, 1, ints(table), ints(start), ints(cu), cu[-1])
    hk, hv = w4.kv_gather(c, 1, ints(table), ints(start), ints(cu), cu[-1], dtype=torch.bfloat16)
    for got, half, which in ((gk, hk, 0), (gv, hv, 1)):
        exp = torch.zeros((cu[-1], heads, D))
        for b in range(7):
            for p in range(new[b]):
                j = (start[b] + p) // ps
                if start[b] >= 0 and j < W and 0 <= table[b][j] < 40:
                    at = (1, table[b][j], slice(None), (start[b] + p) % ps)
                    exp[cu[b] + p] = want[which][at].float()
                    if kv == "int8":
                        exp[cu[b] + p] *= want[2 + which][at][:, None]
        assert torch.equal(got.cpu(), exp)
        assert torch.equal(half.cpu(), exp.bfloat16())


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("B", [1, 2, 65, 300])
def test_append_one_token_each(w4, B, kv):
    """cu None: row b is sequence b's token; slots that take none are skipped."""
    c = random_pool(w4, 1, B + 2, 2, 16, 64, kv, 4)
    table = torch.randperm(B + 2, generator=torch.Generator().manual_seed(5))[:B].int().cuda()[:, None]
    start = ints([i % 16 if i % 5 else -1 for i in range(B)])
    k, v = (torch.randn((B, 2, 64)).cuda() for _ in range(2))
    want = plain_append(c, 0, k, v, table, start, list(range(B + 1)))
    w4.kv_append(c, 0, k, v, table.contiguous(), start)
    for a, b in zip(arrays(c), want):
        assert torch.equal(bits(a.cpu()), bits(b))


def test_append_many_sequences(w4):
    """More sequences than one step of the search over cu."""
    B = 5000
    r = random.Random(6)
    new = [r.choice([0, 0, 1, 2, 3]) for _ in range(B)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    c = random_pool(w4, 1, B, 1, 16, 16, "bf16", 7)
    k, v = (torch.randn((cu[-1], 1, 16)).cuda() for _ in range(2))
    table = ints(r.sample(range(B), B))[:, None].contiguous()
    start = ints([r.randrange(13) for _ in range(B)])
    want = plain_append(c, 0, k, v, table, start, cu)
    w4.kv_append(c, 0, k, v, table, start, ints(cu))
    for a, b in zip(arrays(c), want):
        assert torch.equal(bits(a.cpu()), bits(b))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_append_strides(w4, dt, kv):
    """K and V inside a joint projection's rows, at any alignment."""
    c = random_pool(w4, 1, 8, 2, 16, 64, kv, 8)
    d = random_pool(w4, 1, 8, 2, 16, 64, kv, 8)
    for width, off in ((640, 256), (641, 257), (643, 3)):
        flat = torch.randn((20, width)).to(dt).cuda()
        k = flat[:, off:off + 128].unflatten(1, (2, 64))
        v = flat[:, off + 128:off + 256].unflatten(1, (2, 64))
        table, start, cu = ints([[3, 1], [5, 7]]), ints([9, 2]), ints([0, 12, 20])
        w4.kv_append(c, 0, k, v, table, start, cu)
        w4.kv_append(d, 0, k.contiguous(), v.contiguous(), table, start, cu)
        for a, b in zip(arrays(c), arrays(d)):
            assert torch.equal(bits(a), bits(b))


def test_append_quantizes_like_the_activation_quantizer(w4):
    """The same codes and scales but for the scale's last bit, which can move a
    code where the quotient is next to a half."""
    x = (torch.randn((50, 128)) * torch.logspace(-3, 3, 50)[:, None]).cuda()
    c = w4.KVCache.empty(1, 4, 1, 16, 128, torch.int8)
    w4.kv_append(c, 0, x[:, None], x[:, None], ints([[2, 0, 3, 1]]), ints([0]), ints([0, 50]))
    q, s = w4.a8_quantize_act(x)
    pages = torch.tensor([2, 0, 3, 1]).cuda()
    codes = c.k[0, pages, 0].reshape(64, 128)[:50]
    scales = c.v_scale[0, pages, 0].reshape(64)[:50]
    assert bool(((scales - s).abs() <= s * 2.0 ** -23).all())
    t = x.double() / s.double()[:, None]
    near = ((t - t.floor()) - 0.5).abs() < 1e-4
    assert torch.equal(codes[~near], q[~near])
    assert bool(((codes.int() - q.int()).abs() <= 1).all())


@pytest.mark.parametrize("kv_in", [torch.bfloat16, torch.float32])
def test_append_ties(w4, kv_in):
    """Values at half codes: bf16 rows of few distinct values, bit for bit."""
    g = torch.Generator().manual_seed(9)
    x = torch.randint(-8, 9, (600, 2, 64), generator=g).float().div(16).to(kv_in).cuda()
    c = random_pool(w4, 1, 40, 2, 16, 64, "int8", 10)
    table = torch.randperm(40, generator=g)[:38].int().cuda()[None].contiguous()
    want = plain_append(c, 0, x, x, table, ints([0]), [0, 600])
    w4.kv_append(c, 0, x, x, table, ints([0]), ints([0, 600]))
    for a, b in zip(arrays(c), want):
        assert torch.equal(bits(a.cpu()), bits(b))


# -------------------------------------------------------------- page moves
class Host:
    """The bookkeeping's host form."""

    def __init__(self, table, lens, refs, ps):
        self.t, self.n, self.r, self.ps = [list(x) for x in table], list(lens), list(refs), ps

    def free_pages(self):
        return [p for p, r in enumerate(self.r) if r == 0]

    def reserve(self, add):
        S, W, ok, used = len(self.t), len(self.t[0]), [], 0
        free = self.free_pages()
        at = 0
        for s in range(S):
            end = -(-(self.n[s] + add[s]) // self.ps)
            if add[s] <= 0:
                ok.append(1)
                continue
            if self.n[s] < 0 or end > W:
                ok.append(0)
                continue
            j = self.n[s] // self.ps
            while j < end and self.t[s][j] >= 0:
                j += 1
            used += end - j
            if end > j and used > len(free):
                ok.append(0)
                continue
            ok.append(1)
            for jj in range(j, end):
                self.t[s][jj] = free[at]
                self.r[free[at]] = 1
                at += 1
        return ok

    def fork(self, parents, children):
        S, W, ps = len(self.t), len(self.t[0]), self.ps
        free, used, ok, moves, seen = self.free_pages(), 0, [], [], set()
        t0, n0 = [list(x) for x in self.t], list(self.n)
        for p, c in zip(parents, children):
            good = 0 <= p < S and 0 <= c < S and n0[c] == 0 and t0[c][0] == -1
            src = -1
            if good:
                good = n0[p] >= 0 and -(-n0[p] // ps) <= W
                if good and n0[p] % ps:
                    src = t0[p][n0[p] // ps]
                    good = 0 <= src < len(self.r)
            if good and c in seen:
                good = False
            if not good:
                ok.append(0)
                continue
            seen.add(c)
            used += src >= 0
            if used > len(free):
                ok.append(0)
                continue
            ok.append(1)
            full = n0[p] // ps
            row = t0[p][:full] + ([free[used - 1]] if src >= 0 else [])
            self.t[c] = row + [-1] * (W - len(row))
            self.n[c] = n0[p]
            for x in row:
                if 0 <= x < len(self.r):
                    self.r[x] += 1
            if src >= 0:
                moves.append((src, row[-1]))
        return ok, moves

    def free(self, slots):
        for s in slots:
            if 0 <= s < len(self.t):
                for x in self.t[s]:
                    if 0 <= x < len(self.r):
                        self.r[x] -= 1
                self.t[s] = [-1] * len(self.t[s])
                self.n[s] = 0

    def compact(self):
        live = [p for p, r in enumerate(self.r) if r > 0]
        n = len(live)
        src = [p for p in live if p >= n]
        dst = [p for p in range(n) if self.r[p] <= 0]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.r[d], self.r[s] = self.r[s], 0
        self.t = [[to.get(x, x) if 0 <= x < len(self.r) else -1 for x in row] for row in self.t]
        return n, list(zip(src, dst))

    def same(self, table, refs, lens=None):
        assert table.tolist() == self.t
        assert refs.tolist() == self.r
        assert lens is None or lens.tolist() == self.n


def moved(pools, moves):
    out = [p.clone() for p in pools]
    for s, d in moves:
        for o, p in zip(out, pools):
            o[:, d] = p[:, s]
    return out


def random_state(S, W, ps, pages, seed, empty=0.3):
    """Rows of distinct pages, some empty, some pages held twice."""
    r = random.Random(seed)
    order = r.sample(range(pages), pages)
    table, lens, refs = [], [], [0] * pages
    for s in range(S):
        room = min(W, len(order))
        k = 0 if r.random() < empty else r.randint(0, room)
        row = [order.pop() for _ in range(k)]
        for x in row:
            refs[x] += 1
        lens.append(0 if not k else r.randint((k - 1) * ps + 1, k * ps))
        table.append(row + [-1] * (W - k))
    return table, lens, refs


@pytest.mark.parametrize("S,W,ps,pages", [(1, 1, 16, 1), (4, 6, 16, 30), (40, 8, 32, 200),
                                          (3, 2000, 16, 5000), (1500, 4, 64, 4000), (2500, 2, 16, 100)])
def test_reserve(w4, S, W, ps, pages):
    r = random.Random(S)
    table, lens, refs = random_state(S, W, ps, pages, 10 + S)
    h = Host(table, lens, refs, ps)
    t, n, f = ints(table), ints(lens), ints(refs)
    for step in range(3):
        add = [r.choice([0, 1, 1, -2, ps, 3 * ps + 1, W * ps, 2 ** 31 - 1]) for _ in range(S)]
        ok = w4.kv_reserve(t, n, f, ints(add), ps)
        assert ok.tolist() == h.reserve(add)
        h.same(t, f, n)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("S,W,ps,pages,n", [(2, 3, 16, 8, 1), (12, 6, 16, 60, 9), (300, 5, 16, 700, 200),
                                            (64, 4, 32, 40, 70), (2600, 2, 16, 3000, 2300)])
def test_fork_and_free(w4, S, W, ps, pages, n, kv):
    r = random.Random(S + n)
    table, lens, refs = random_state(S, W, ps, pages, 20 + S, empty=0.5)
    lens[0] = lens[0] or 5 if table[0][0] >= 0 else 0
    c = random_pool(w4, 2, pages, 1, ps, 16, kv, 21)
    h = Host(table, lens, refs, ps)
    t, ln, f = ints(table), ints(lens), ints(refs)
    for step in range(3):
        parents = [r.randrange(-1, S + 1) for _ in range(n)]
        empty = [s for s in range(S) if h.n[s] == 0 and h.t[s][0] == -1] or [0]
        children = [r.choice(empty) if r.random() < 0.9 else r.randrange(-1, S + 1) for _ in range(n)]
        before = arrays(c)
        ok, moves = h.fork(parents, children)
        want = moved([x.cpu() for x in before], moves)
        got = w4.kv_fork(c, t, ln, f, ints(parents), ints(children))
        assert got.tolist() == ok
        h.same(t, f, ln)
        for a, b in zip(arrays(c), want):
            assert torch.equal(bits(a.cpu()), bits(b))
        gone = [r.randrange(-2, S + 2) for _ in range(max(1, S // 4))]
        gone += gone[:2]
        w4.kv_free(t, ln, f, ints(gone))
        h.free(dict.fromkeys(gone))
        h.same(t, f, ln)


def test_fork_reserved_pages_stay(w4):
    """Pages reserved beyond a parent's length are not the child's."""
    c = random_pool(w4, 1, 6, 1, 16, 16, "bf16", 22)
    t, n, f = ints([[4, 2, 0], [-1, -1, -1]]), ints([20, 0]), ints([1, 0, 1, 0, 1, 0])
    assert w4.kv_fork(c, t, n, f, ints([0]), ints([1])).tolist() == [1]
    assert t.tolist() == [[4, 2, 0], [4, 1, -1]]
    assert f.tolist() == [1, 1, 1, 0, 2, 0] and n.tolist() == [20, 20]
    assert torch.equal(c.k[:, 1], c.k[:, 2])


@pytest.mark.parametrize("kv", ["bf16", "int8"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,W,ps,pages", [(1, 1, 16, 1), (4, 6, 16, 30), (40, 8, 32, 300),
                                          (1500, 3, 16, 5000), (3, 4, 16, 2049)])
def test_compact(w4, S, W, ps, pages, in_place, kv):
    table, lens, refs = random_state(S, W, ps, pages, 30 + S)
    table[0][-1] = pages + 3  # an entry that is no page
    c = random_pool(w4, 2, pages, 1, ps, 16, kv, 31)
    h = Host(table, lens, refs, ps)
    t, f = ints(table), ints(refs)
    pools = [x.cpu() for x in arrays(c)]
    n, moves = h.compact()
    to, fo = (None, None) if in_place else (torch.empty_like(t), torch.empty_like(f))
    rt, rf, live = w4.kv_compact(c, t, f, table_out=to, refs_out=fo)
    assert live.tolist() == [n]
    h.same(rt, rf)
    if in_place:
        assert rt is t and rf is f
    else:
        assert t.tolist() == table and f.tolist() == refs
    for a, b in zip(arrays(c), moved(pools, moves)):
        assert torch.equal(bits(a.cpu()), bits(b))
    # a second call has nothing to move
    pools = [x.cpu() for x in arrays(c)]
    rt2, rf2, live2 = w4.kv_compact(c, rt, rf)
    assert live2.tolist() == [n]
    h.same(rt2, rf2)
    for a, b in zip(arrays(c), pools):
        assert torch.equal(bits(a.cpu()), bits(b))


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_copy_pages(w4, kv):
    """To another cache; pairs with a page outside are skipped."""
    a = random_pool(w4, 3, 20, 2, 32, 48, kv, 40)
    b = random_pool(w4, 3, 9, 2, 32, 48, kv, 41)
    src, dst = [3, 19, 20, -1, 7, 7], [0, 8, 1, 2, 9, 4]
    want = [x.clone() for x in arrays(b)]
    for s, d in zip(src, dst):
        if 0 <= s < 20 and 0 <= d < 9:
            for w, x in zip(want, arrays(a)):
                w[:, d] = x[:, s]
    w4.kv_copy_pages(b, ints(dst), a, ints(src))
    for x, w in zip(arrays(b), want):
        assert torch.equal(bits(x), bits(w))


def test_moves_in_a_large_pool(w4):
    """Page offsets that pass 32 bits."""
    c = w4.KVCache.empty(2, 20000, 8, 64, 128, torch.bfloat16)
    c.k[:, 19999] = 3.0
    c.v[:, 19999] = 4.0
    refs = torch.zeros(20000, dtype=torch.int32, device="cuda")
    refs[19999] = 1
    t, f, live = w4.kv_compact(c, ints([[19999, -1]]), refs)
    assert t.tolist() == [[0, -1]] and live.item() == 1 and int(f[0]) == 1 and int(f.sum()) == 1
    assert bool((c.k[:, 0] == 3.0).all()) and bool((c.v[:, 0] == 4.0).all())


def test_moves_in_a_graph(w4):
    """Fork, free and compact captured once and replayed."""
    table, lens, refs = random_state(12, 6, 16, 90, 50, empty=0.0)
    table += [[-1] * 6 for _ in range(4)]
    lens += [0] * 4
    c = random_pool(w4, 2, 90, 1, 16, 16, "bf16", 51)
    t, n, f = ints(table), ints(lens), ints(refs)
    keep = [x.clone() for x in (t, n, f, c.k, c.v)]
    par, kid, ok = ints([0, 3, 3, 7]), ints([12, 13, 14, 15]), ints([0] * 4)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    live = ints([0])

    def step():
        w4.kv_fork(c, t, n, f, par, kid, ok=ok, workspace=ws)
        w4.kv_free(t, n, f, par[:1])
        w4.kv_compact(c, t, f, live=live, workspace=ws)

    step()
    want = [x.clone() for x in (t, n, f, c.k, c.v, ok, live)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        for x, y in zip((t, n, f, c.k, c.v), keep):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((t, n, f, c.k, c.v, ok, live), want):
            assert torch.equal(x, y)
