"""AdamW with 8-bit states on the GPU against its definition in 64 bits.

Tolerances.  Moments are computed in binary64, where a few roundings leave
8 * 2^-53 of their terms: a scale is their largest, rounded once to binary32
(two neighbours where the rounding is undecided), and a code's root is within
1/2 of the value's, and 1e-9 for what 255 times those roundings leave.  The
weights take the moments rounded once to binary32, a division, a root, and two
products more: 16 F32 of the update and 4 F32 of the weight.
"""
import pytest
import torch

import sgd_gradient_all_amd as ddl

pytestmark = pytest.mark.gpu

F32 = torch.finfo(torch.float32).eps / 2
T = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
B = 256
SPANS = [(0, 1), (3, 5), (16, 4096), (5000, 2047), (9001, 1), (9010, 0), (9016, 3), (9020, 256),
         (9276, 257), (9600, 4097), (14000, 1024)]
SIZE = 15100


def normal(g, n, sigma=1.0, dtype=torch.float32):
    return (torch.randn(n, generator=g, device="cuda") * sigma).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def blocks_of(spans):
    """[(slice of the elements, index of the block)]"""
    out = []
    for o, c in spans:
        for b in range(0, c, B):
            out.append((slice(o + b, o + min(b + B, c)), len(out)))
    return out


def states(g, size, blocks, first=0):
    m = torch.randint(-127, 128, (size + first,), generator=g, device="cuda").to(torch.int8)
    v = torch.randint(1, 256, (size + first,), generator=g, device="cuda").to(torch.uint8)
    ms, vs = normal(g, blocks, 1e-2).abs() + 1e-4, normal(g, blocks, 1e-2).square() + 1e-6
    return [m[first:], v[first:], ms, vs]


def decoded(m, v, ms, vs):
    k, h = m.double(), v.double() / 255
    return k * k.abs() / 127 ** 2 * ms.double(), h ** 4 * vs.double()


def check_codes(k, scale, want, top, power, exact=True):
    """Codes k of the values want (64 bits) under scale."""
    assert float((scale.double() - want.abs().max()).abs()) <= 1.01 * F32 * float(want.abs().max())
    if float(scale) == 0:
        assert (k == 0).all()
        return
    root = top * (want.abs() / scale.double()) ** (1 / power)
    low = (root < 0.5) & (want != 0) if power == 4 else torch.zeros_like(root, dtype=torch.bool)
    d = (k.double().abs() - root).abs()
    assert (d[~low] <= 0.5 + 1e-9).all() and (k[low] == 1).all()
    assert ((k == 0) | (torch.sign(k.double()) == torch.sign(want))).all()


@pytest.mark.parametrize("grad,copy,replicas", [("f32", None, 1), ("f16", "f16", 1),
                                                ("bf16", "bf16", 3), ("f32", "bf16", 2)])
@pytest.mark.parametrize("offset", [0, 1])
def test_step(grad, copy, replicas, offset):
    h = ddl.AdamW8(SPANS)
    parts = blocks_of(SPANS)
    assert h.blocks == len(parts)
    g_ = gen(1 + offset)
    gr = normal(g_, SIZE + offset, 1e-2, T[grad])[offset:]
    w = normal(g_, SIZE + offset, 0.02)[offset:]
    st = states(g_, SIZE, h.blocks, offset)
    ws = [w.clone() for _ in range(replicas)]
    cp = torch.full((SIZE,), 5.0, device="cuda", dtype=T[copy]) if copy else None
    inside = torch.zeros(SIZE, device="cuda", dtype=torch.bool)
    for o, c in SPANS:
        inside[o:o + c] = True
    before = [t.clone() for t in st]
    lr, b1, b2, eps, wd, step = 2e-3, 0.9, 0.95, 1e-8, 0.1, 3
    print(f"adamw8 {grad} {copy} {replicas} {offset}", flush=True)
    h.step(gr, *st, ws, lr=lr, beta1=b1, beta2=b2, eps=eps, weight_decay=wd, step=step, copy=cp)
    values = [torch.full((SIZE,), 7.0, device="cuda") for _ in range(2)]
    h.values(*st, *values)
    for at, b in parts:
        m, v = decoded(before[0][at], before[1][at], before[2][b], before[3][b])
        gd = gr[at].double()
        mag = b1 * m.abs() + (1 - b1) * gd.abs()
        m, v = b1 * m + (1 - b1) * gd, b2 * v + (1 - b2) * gd * gd
        check_codes(st[0][at], st[2][b], m, 127, 2)
        check_codes(st[1][at], st[3][b], v, 255, 4)
        hat = (v / (1 - b2 ** step)).sqrt() + eps
        want = w[at].double() * (1 - lr * wd) - lr * (m / (1 - b1 ** step)) / hat
        big = lr * (mag / (1 - b1 ** step)) / hat
        assert ((ws[0][at].double() - want).abs()
                <= 16 * F32 * big + 4 * F32 * w[at].double().abs()).all()
        for got, want in zip(values, decoded(st[0][at], st[1][at], st[2][b], st[3][b])):
            assert ((got[at].double() - want).abs() <= 1.01 * F32 * want.abs() + 2e-45).all()
    for t, t0 in ((st[0], before[0]), (st[1], before[1])):
        assert torch.equal(t[~inside], t0[~inside])
    assert torch.equal(ws[0][~inside], w[~inside])
    assert all((x[~inside] == 7.0).all() for x in values)
    for k in ws[1:]:
        assert torch.equal(k[inside], ws[0][inside]) and torch.equal(k[~inside], w[~inside])
    if copy:
        assert torch.equal(cp[inside], ws[0][inside].to(T[copy]))
        assert (cp[~inside] == 5.0).all()


def test_first_steps_follow_the_definition():
    """From zeros, step by step; codes are decoded, so that steps do not add up."""
    spans = [(0, 700), (704, 300)]
    h, parts, g_ = ddl.AdamW8(spans), blocks_of(spans), gen(3)
    st = [torch.zeros(1004, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.zeros(h.blocks, device="cuda") for _ in range(2)]
    w = normal(g_, 1004, 0.02)
    for step in range(1, 6):
        gr = normal(g_, 1004, 1e-2)
        gr[10:20] = 0.0
        before, w0 = [t.clone() for t in st], w.double()
        h.step(gr, *st, [w], lr=1e-2, beta1=0.9, beta2=0.999, step=step)
        for at, b in parts:
            m, v = decoded(before[0][at], before[1][at], before[2][b], before[3][b])
            m, v = 0.9 * m + 0.1 * gr[at].double(), 0.999 * v + 0.001 * gr[at].double() ** 2
            check_codes(st[0][at], st[2][b], m, 127, 2)
            check_codes(st[1][at], st[3][b], v, 255, 4)
            up = 1e-2 * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.999 ** step)).sqrt() + 1e-8)
            # m's terms may cancel: 4 F32 of them, 0.1 |g| and the state's 1e-2 at most
            slack = 16 * F32 * (up.abs() + 1e-2 * 0.02 / ((v / (1 - 0.999 ** step)).sqrt() + 1e-8))
            assert ((w[at].double() - (w0[at] - up)).abs()
                    <= slack + 4 * F32 * w0[at].abs()).all()


@pytest.mark.parametrize("b1,b2", [(0.9, 0.95), (0.8, 0.999)])
def test_scales_between_two_binary32_numbers(b1, b2):
    """0.9 s + 0.1 g is often midway: it goes by the last bit of the formula's sum in
    64 bits, term by term."""
    blocks = 20000
    g_, n = gen(12), blocks * B
    h = ddl.AdamW8([(0, n)])
    st = states(g_, n, blocks)
    st[0][::B], st[1][::B] = 127, 255
    gr = normal(g_, n, 1e-3, torch.float16)
    gr[::B] = normal(g_, blocks, 1e-2, torch.float16).abs()
    before, w = [t.clone() for t in st], torch.zeros(n, device="cuda")
    h.step(gr, *st, [w], lr=1e-2, beta1=b1, beta2=b2, step=9)
    g = gr.double()
    m, v = (x.view(blocks, B) for x in (before[0].double(), before[1].double()))
    m = b1 * (m * m.abs() / 127 ** 2 * before[2].double()[:, None]) + (1 - b1) * g.view(blocks, B)
    v = b2 * ((v / 255) ** 4 * before[3].double()[:, None]) + (1 - b2) * (g * g).view(blocks, B)
    top = m.abs().amax(1)
    # the 29 bits behind binary32's: a half and at most 4 last bits of binary64 beside
    rest = (top.view(torch.int64) & ((1 << 29) - 1)) - (1 << 28)
    assert int((rest.abs() <= 4).sum()) > 100 or b1 != 0.9
    assert torch.equal(st[2], top.float())
    # (1 - b2) g g may be rounded in another order: where that is not near a half
    rest = (v.amax(1).view(torch.int64) & ((1 << 29) - 1)) - (1 << 28)
    assert torch.equal(st[3][rest.abs() > 4], v.amax(1).float()[rest.abs() > 4])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite_gradients_spoil_their_block_alone(bad):
    h = ddl.AdamW8([(0, 1024)])
    g_ = gen(4)
    st = states(g_, 1024, 4)
    clean = [t.clone() for t in st]
    gr, w = normal(g_, 1024), normal(g_, 1024)
    w2 = w.clone()
    h.step(gr, *clean, [w2], lr=1e-2)
    gr[300] = bad
    h.step(gr, *st, [w], lr=1e-2)
    m, v = torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    h.values(*st, m, v)
    assert torch.isnan(m[256:512]).all() and torch.isnan(v[256:512]).all()
    others = torch.ones(1024, device="cuda", dtype=torch.bool)
    others[256:512] = False
    for a, b in zip(st[:2], clean[:2]):
        assert torch.equal(a[others], b[others])
    others[256:512] = True
    others[300] = False
    assert torch.equal(w[others], w2[others])  # this step's own weights
    h.step(torch.zeros_like(gr), *st, [w], lr=1e-2, step=2)
    assert torch.isnan(w[256:512]).all() and torch.isfinite(w[512:]).all()


def test_extremes_of_a_block():
    """Values far under the largest: m goes to 0, v keeps its least code; a block
    of zeros keeps scales of 0; huge and tiny gradients."""
    h, b2 = ddl.AdamW8([(0, 1024)]), 0.999
    st = [torch.zeros(1024, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.full((4,), 3.0, device="cuda") for _ in range(2)]
    st[2][1] = st[3][1] = 0.0
    gr, w = torch.full((1024,), 1e-12, device="cuda"), torch.zeros(1024, device="cuda")
    gr[0] = 1.0
    gr[256:512] = 0.0
    gr[512:768] = 1e18      # squares stay inside binary32
    gr[768:] = 1e-30        # and leave it
    h.step(gr, *st, [w], lr=1e-2, beta2=b2)
    assert (st[0][1:256] == 0).all() and (st[1][1:256] == 1).all()
    assert int(st[0][0]) == 127 and int(st[1][0]) == 255
    assert (st[0][256:512] == 0).all() and (st[1][256:512] == 0).all()
    assert float(st[2][1]) == 0 and float(st[3][1]) == 0
    assert (st[0][512:] == 127).all() and (st[1][512:768] == 255).all()
    assert float(st[3][3]) == 0 and (st[1][768:] == 0).all()
    assert torch.isfinite(w).all() and (w[256:512] == 0).all()


def test_same_bits_on_another_stream_and_in_a_graph():
    h, g_ = ddl.AdamW8(SPANS), gen(5)
    gr, w0 = normal(g_, SIZE, 1e-2), normal(g_, SIZE, 0.02)
    start = states(g_, SIZE, h.blocks)

    def fresh():
        return [t.clone() for t in start] + [w0.clone()]

    eager = fresh()
    want = []
    for step in range(3):
        h.step(gr, *eager[:4], [eager[4]], lr=1e-2, step=1)
        want.append([t.clone() for t in eager])
    side, s = fresh(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for step in range(3):
        h.step(gr, *side[:4], [side[4]], lr=1e-2, step=1, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(side, want[step]))
    held, graph = fresh(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        h.step(gr, *held[:4], [held[4]], lr=1e-2, step=1, stream=s)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[step])), step
        (torch.randn(64, 64, device="cuda") @ torch.randn(64, 64, device="cuda")).sum().item()


def test_first_call_in_a_capture_is_refused():
    h = ddl.AdamW8([(0, 8)])
    st = [torch.zeros(8, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.zeros(1, device="cuda") for _ in range(2)]
    v = [torch.zeros(8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        v[0].add_(1)
        with pytest.raises(ddl.DDLError) as e:
            h.step(v[0], *st, [v[1]], lr=1e-3, stream=s)
        assert e.value.code == -9
        with pytest.raises(ddl.DDLError) as e:
            h.values(*st, v[0], v[1], stream=s)
    assert e.value.code == -9


def test_offsets_past_32_bits():
    """A span behind 2^32 elements."""
    size = (1 << 32) + 5000
    h, g_ = ddl.AdamW8([(5, 300), (size - 1000, 1000)]), gen(6)
    small = ddl.AdamW8([(0, 300), (300, 1000)])
    one = states(g_, 1300, 6)
    gr, w = normal(g_, 1300, 1e-2, torch.float16), normal(g_, 1300, 0.02)

    def spread(t):
        big = torch.zeros(size, device="cuda", dtype=t.dtype)
        big[5:305], big[size - 1000:] = t[:300], t[300:]
        return big

    big = [spread(t) for t in one[:2]] + [t.clone() for t in one[2:]]
    bgr, bw = spread(gr), spread(w)
    print("adamw8 past 32 bits", flush=True)
    h.step(bgr, *big, [bw], lr=1e-2)
    small.step(gr, *one, [w], lr=1e-2)
    for a, b in ((big[0], one[0]), (big[1], one[1]), (bw, w)):
        assert torch.equal(a[5:305], b[:300]) and torch.equal(a[size - 1000:], b[300:])
    assert torch.equal(big[2], one[2]) and torch.equal(big[3], one[3])
    assert int((bw != 0).sum()) <= 1300


def test_training_with_8_bit_states_follows_binary32():
    """200 steps on a quadratic: 8-bit and binary32 states take the weights to
    the same place, within a tenth of the way."""
    n, g_ = 4096, gen(7)
    goal = normal(g_, n)
    adam, adam8 = ddl.AdamW([(0, n)]), ddl.AdamW8([(0, n)])
    w, w8 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    st = [torch.zeros(n, device="cuda", dtype=t) for t in (torch.int8, torch.uint8)] \
        + [torch.zeros(adam8.blocks, device="cuda") for _ in range(2)]
    for step in range(1, 201):
        adam.step(w - goal, m, v, [w], lr=1e-2, step=step)
        adam8.step(w8 - goal, *st, [w8], lr=1e-2, step=step)
    assert float((w8 - w).norm()) <= 0.1 * float(w.norm())
