"""The operators around the 4-bit layers run together, as in a transformer
block whose projections are 8-bit: norm -> QKV -> rotary positions in place ->
output projection into the residual stream -> norm -> MLP -> residual stream,
and the rotary table inside the 4-bit QKV layer.  Every stage is checked
against the fp64 formula of its actual inputs (tolerances: the operators' own
test files derive them), eagerly and replayed from a captured graph."""
import numpy as np
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq
from bit_diffusion_transformer_w4a4_b200 import workloads as W

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HALF = 2.0 ** -8          # half a step of bf16
BF = torch.bfloat16


def _weight(N, K, out, seed):
    """A linear's 8-bit weight, quantised row by row by the library itself."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5
    codes = torch.empty(N, K, dtype=out, device="cuda")
    scales = torch.empty(N, device="cuda")
    svdq.rms_quantize8(w, codes, scales, norm=False)
    step = 0.5 if out == torch.int8 else 2.0 ** -4
    err = (codes.double() * scales.double()[:, None] - w.double()).abs()
    ref = scales.double()[:, None] if out == torch.int8 else w.double().abs() + 2.0 ** -6 * scales.double()[:, None]
    assert (err <= step * 1.001 * ref).all()
    return codes, scales


class Block:
    def __init__(self, S, hidden, heads, mlp, out, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
        self.S, self.H, self.heads, self.out = S, hidden, heads, out
        self.D = hidden // heads
        self.x = r(S, hidden)
        self.stream = self.x.clone()
        self.n1, self.n2 = (1 + 0.2 * r(hidden)).to(BF), (1 + 0.2 * r(hidden)).to(BF)
        images = min(S, 2)
        self.g1, self.g2 = r(images, hidden), r(images, hidden)
        self.b = {k: 0.1 * r(n) for k, n in (("qkv", 3 * hidden), ("o", hidden), ("fc1", mlp), ("fc2", hidden))}
        self.w = {"qkv": _weight(3 * hidden, hidden, out, 1), "o": _weight(hidden, hidden, out, 2),
                  "fc1": _weight(mlp, hidden, out, 3), "fc2": _weight(hidden, mlp, out, 4)}
        self.rope = svdq.RopeAxes(self.D, [self.D // 4, self.D // 4, self.D // 2])
        self.pos = torch.randint(0, 512, (S, 3), generator=g, device="cuda", dtype=torch.int32)
        e = lambda n, t=BF: torch.empty(S, n, dtype=t, device="cuda")  # noqa: E731
        self.c = {k: (e(n, out), torch.empty(S, device="cuda")) for k, n in
                  (("qkv", hidden), ("o", hidden), ("fc1", hidden), ("fc2", mlp))}
        self.qkv, self.qkv_raw, self.attn, self.mid, self.hid = e(3 * hidden), e(3 * hidden), e(hidden), e(hidden), e(mlp)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dense(self, k, y, **kw):
        (a, sa), (w, sw) = self.c[k], self.w[k]
        svdq.dense_forward(a, w, y, a_scale=sa, w_scale=sw, bias=self.b[k], device_error=self.err, **kw)

    def run(self):
        half = -(-self.S // 2)
        self.stream.copy_(self.x)
        svdq.rms_quantize8(self.stream, *self.c["qkv"], weight=self.n1)
        self.dense("qkv", self.qkv)
        self.qkv_raw.copy_(self.qkv)
        heads = self.qkv.view(self.S, 3, self.heads, self.D)
        self.rope.apply(heads[:, 0], self.pos, k=heads[:, 1])
        self.attn.copy_(self.qkv[:, 2 * self.H:])             # the attention itself is the caller's
        svdq.rms_quantize8(self.attn, *self.c["o"], norm=False)
        self.dense("o", self.mid, gate=self.g1, gate_rows=half)
        # the residual's addition inside the norm, and inside the linear
        svdq.rms_quantize8(self.mid, *self.c["fc1"], residual=self.stream, h=self.stream, weight=self.n2)
        self.dense("fc1", self.hid, act="gelu")
        svdq.rms_quantize8(self.hid, *self.c["fc2"], norm=False)
        self.before = None
        self.kept = self.stream.clone()
        self.dense("fc2", self.stream, gate=self.g2, gate_rows=half, residual=self.stream)

    def check_codes(self, k, v):
        """codes * scale against v (fp64): half a code step."""
        q, s = self.c[k]
        s = s.double()[:, None]
        step = 0.5 * s if self.out == torch.int8 else torch.clamp(v.abs() * 2.0 ** -4, min=1e-30) + s * 2.0 ** -10
        assert ((q.double() * s - v).abs() <= step * 1.001 + 2.0 ** -17 * v.abs()).all(), k

    def check_dense(self, k, y, act=False, gate=None, res=None):
        (a, sa), (w, sw) = self.c[k], self.w[k]
        acc = (a.double() @ w.double().t()) * sa.double()[:, None] * sw.double()[None]
        mag = (a.double().abs() @ w.double().abs().t()) * sa.double()[:, None] * sw.double()[None]
        steps = 0 if self.out == torch.int8 else -(-a.shape[1] // 16)
        v = acc + self.b[k].double()
        err = 1.2 * (mag * steps * 2.0 ** -22 + (v.abs() + self.b[k].double().abs()) * 2.0 ** -19)
        if act:
            v = 0.5 * v * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
        if gate is not None:
            g = gate.double().repeat_interleave(-(-self.S // 2), 0)[:self.S]
            v, err = v * g, err * g.abs()
        if res is not None:
            v, err = v + res.double(), err + res.double().abs() * 2.0 ** -23
        assert ((y.double() - v).abs() <= HALF * v.abs() + err + 1e-30).all(), k

    def check(self):
        norm = lambda h, w: h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * w.double()  # noqa: E731
        self.check_codes("qkv", norm(self.x.double(), self.n1))
        self.check_dense("qkv", self.qkv_raw)
        f = torch.cat([10000.0 ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d) for d in self.rope.axis_dims])
        axis = torch.cat([torch.full((d // 2,), a, device="cuda") for a, d in enumerate(self.rope.axis_dims)])
        ang = (self.pos.double()[:, axis] * f)[:, None]
        raw = self.qkv_raw.double().view(self.S, 3, self.heads, self.D)
        got = self.qkv.double().view(self.S, 3, self.heads, self.D)
        for i in (0, 1):
            a, b = raw[:, i, :, 0::2], raw[:, i, :, 1::2]
            for o, v in ((0, a * torch.cos(ang) - b * torch.sin(ang)), (1, a * torch.sin(ang) + b * torch.cos(ang))):
                assert ((got[:, i, :, o::2] - v).abs() <= HALF * v.abs() + 2.0 ** -20 * (a.abs() + b.abs())).all()
        assert torch.equal(raw[:, 2], got[:, 2])
        self.check_codes("o", self.attn.double())
        self.check_dense("o", self.mid, gate=self.g1)
        h = (self.mid.float() + self.x.float()).to(BF)
        assert torch.equal(h, self.kept)
        self.check_codes("fc1", norm(h.double(), self.n2))
        self.check_dense("fc1", self.hid, act=True)
        self.check_codes("fc2", self.hid.double())
        self.check_dense("fc2", self.stream, gate=self.g2, res=h)
        assert self.err.item() == 0


@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("S,hidden,heads,mlp", [(1, 512, 4, 2048), (77, 768, 6, 3088), (601, 1536, 12, 6144), (2500, 1024, 8, 4096)])
def test_block(S, hidden, heads, mlp, out):
    b = Block(S, hidden, heads, mlp, out)
    b.run()
    torch.cuda.synchronize()
    b.check()
    first = b.stream.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    b.stream.zero_(), b.qkv.zero_(), b.hid.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, b.stream)


def test_two_blocks_on_two_streams():
    """Nothing is shared between calls: two chains on two streams at once, and
    two captured graphs replayed at once, give the bits of each alone."""
    blocks = [Block(300, 768, 6, 3072, torch.float8_e4m3fn, seed=i) for i in range(2)]
    want = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        want.append(b.stream.clone())
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(4):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    assert all(torch.equal(w, b.stream) for w, b in zip(want, blocks))
    graphs = []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, b.stream) for w, b in zip(want, blocks))


def test_explicit_stream():
    b = Block(40, 512, 4, 2048, torch.int8)
    s = torch.cuda.Stream()
    y = torch.empty(40, 512, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    svdq.rms_quantize8(b.x, *b.c["o"], norm=False, stream=s.cuda_stream)
    svdq.dense_forward(*[b.c["o"][0], b.w["o"][0], y], a_scale=b.c["o"][1], w_scale=b.w["o"][1], bias=b.b["o"], stream=s.cuda_stream)
    s.synchronize()
    b.check_dense("o", y)


@pytest.mark.parametrize("single_sm", [False, True])
def test_table_in_the_4bit_qkv_layer(single_sm):
    """RopeAxes.table as the rotary table of svdq_linear_forward_qkv: the same
    result as with the table rounded from fp64, to the table's own error."""
    M, H = 300, 2
    lay = W.Layer("qkv", M=M, K=512, N=3 * H * 128, r=32, variant=W.NVFP4, config_id=99, layer_id=7)
    pw = W.synthetic_packed(lay)
    gq, gk, _ = W.qkv_epilogue_inputs(M)
    h = svdq.SVDQWeights(pw, M, qkv_norm=(gq, gk, 1e-6), single_sm=single_sm)
    h.set_deterministic(True)
    x = torch.from_numpy(W.activations(lay).view(np.int16)).cuda().view(BF)
    pos = torch.stack([torch.zeros(M), torch.arange(M) // 16, torch.arange(M) % 16], 1).to(torch.int32).cuda()
    rope = svdq.RopeAxes(128, [16, 56, 56])
    table = torch.empty(M, 128, device="cuda")
    rope.table(pos, table)
    f = torch.cat([10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d) for d in (16, 56, 56)])
    axis = torch.tensor([0] * 8 + [1] * 28 + [2] * 28, device="cuda")
    ang = pos.double()[:, axis] * f
    ref = torch.stack([torch.cos(ang), torch.sin(ang)], -1).reshape(M, 128).float()
    y, z = (torch.empty(M, 3 * H * 128, dtype=BF, device="cuda") for _ in range(2))
    h.linear_forward_qkv(x, table, y, M)
    h.linear_forward_qkv(x, ref, z, M)
    torch.cuda.synchronize()
    assert h.device_status() == 0
    # the tables differ by at most 2^-21 each; the largest element of a head's pair bounds what that moves
    big = z.double().view(M, 3 * H, 64, 2).norm(dim=-1, keepdim=True).expand(-1, -1, -1, 2).reshape(M, -1)
    assert ((y.double() - z.double()).abs() <= 2 * HALF * z.double().abs() + 2.0 ** -19 * big).all()
    h.close()
