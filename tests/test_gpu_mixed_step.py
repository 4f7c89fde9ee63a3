"""The decode step with a token mixer in every layer (q4gemv_run_stack_mixed)
against the chain in 64 bits with the same binary16 roundings, token by token.

Tolerance: between the step's input and output lie six vectors that are rounded
to binary16 (QKV output, rotated queries and keys, mixer, O, gate+up and down
outputs); the 64-bit chain rounds the same vectors, and a rounding that falls
the other way is one step, 2^-10 of its element.  Every product is preceded by
a scale to unit RMS, so a relative change of its input is the same relative
change of its output's RMS: 6 * 2^-10 in the metric of the GEMV tests, plus
their tolerance for the products' own sums (2e-3)."""
import numpy as np
import pytest

import oracle
import synth
from tests import mix_ref as ref
from tests.gpu_util import TOL, bits_of, f16_dev, packed_on_gpu, rel_err

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import q4_quantized_decode_b200 as q4  # noqa: E402

DEV = "cuda:0"
STEP_TOL = 6 * 2.0 ** -10 + TOL


@pytest.fixture(scope="module")
def eng():
    e = q4.Q4Gemv(0)
    yield e
    e.close()


class Trunk:
    """A few layers' matrices, caches and states, on the GPU and for the reference."""

    def __init__(self, eng, kinds, hidden, ffn, hq, hkv, seed, tokens, page=4):
        self.kinds, self.hidden, self.ffn, self.hq, self.hkv = kinds, hidden, ffn, hq, hkv
        self.d = hidden // hq
        self.qkv = hidden + 2 * hkv * self.d
        dims = [(self.qkv, hidden), (hidden, hidden), (2 * ffn, hidden), (hidden, ffn)]
        self.rows = [[synth.q4_0_matrix(seed, synth.weight_id(4 * l + t), *dims[t]) for t in range(4)]
                     for l in range(len(kinds))]
        self.dims = dims
        self.layers = [tuple(packed_on_gpu(eng, r[t], *dims[t]) for t in range(4)) for r in self.rows]
        gen = torch.Generator().manual_seed(seed)
        self.mixers, self.state, self.decay = [], [], []
        for kind in kinds:
            if kind == "attention":
                table, pool = ref.table_of([tokens], page, gen)
                k = torch.full((pool, page, hkv, self.d), float("nan"), dtype=torch.float16, device=DEV)
                self.mixers.append(q4.PagedKV(k, k.clone(), table.to(DEV)))
                self.state.append([[], []])
                self.decay.append(None)
            else:
                g = -torch.rand(hq, generator=gen)
                s = torch.randn(hq, self.d, self.d, generator=gen)
                self.mixers.append((g.to(DEV), s.to(DEV)))
                self.state.append(s.double())
                self.decay.append(g.double())
        self.freqs = eng.rope_freqs(self.d // 2, base=1000.0)

    def step(self, eng, x, n, **kw):
        length = torch.tensor([n], dtype=torch.int32, device=DEV)
        return eng.run_stack_mixed(self.layers, self.mixers, x, self.hidden, self.ffn, self.hq, self.hkv, length,
                                   freqs=self.freqs, **kw)

    def reference(self, x, n):
        """One token through the 64-bit chain; x and the result are f16 bits."""
        d, hkv, hq = self.d, self.hkv, self.hq
        h16 = lambda v: torch.from_numpy(oracle.f16_to_f64(oracle.f64_to_f16(np.asarray(v))))  # noqa: E731
        s = 1.0
        for l, kind in enumerate(self.kinds):
            gemv = lambda t, v, s: oracle.f64_to_f16(  # noqa: E731
                s * oracle.q4_gemv(self.rows[l][t], self.dims[t][1], v.reshape(1, -1), threads=8)[0])
            a = torch.from_numpy(oracle.f16_to_f64(gemv(0, x, s)))
            if kind == "attention":
                pos = torch.tensor([n - 1])
                q = h16(ref.rotate(a[:self.hidden].view(1, hq, d), pos, self.freqs.cpu())[0])[0]
                k = h16(ref.rotate(a[self.hidden:self.hidden + hkv * d].view(1, hkv, d), pos, self.freqs.cpu())[0])[0]
                self.state[l][0].append(k)
                self.state[l][1].append(a[self.hidden + hkv * d:].view(hkv, d))
                ks, vs = torch.stack(self.state[l][0]), torch.stack(self.state[l][1])
                m = torch.cat([ref.attend(q[h:h + 1], ks[:, h * hkv // hq], vs[:, h * hkv // hq], n - 1, d ** -0.5)[0][0]
                               for h in range(hq)])
            else:
                q, k, v = a[:hkv * d].view(hkv, d), a[hkv * d:2 * hkv * d].view(hkv, d), a[2 * hkv * d:].view(hq, d)
                S = self.state[l]
                each = hq // hkv
                for h in range(hq):
                    S[h] = torch.exp(self.decay[l][h]) * S[h] + torch.outer(k[h // each], v[h])
                m = torch.cat([d ** -0.5 * (q[h // each] @ S[h]) for h in range(hq)])
            mb = oracle.f64_to_f16(m.numpy())
            b = gemv(1, mb, oracle.unit_rms_scale(mb))
            u = gemv(2, b, oracle.unit_rms_scale(b))
            w = oracle.swiglu(u.reshape(1, -1))[0]
            ms = float(np.mean(w * w))
            y = (1.0 / np.sqrt(ms) if ms > 0 else 0.0) * oracle.q4_gemv_f64(self.rows[l][3], self.ffn, w.reshape(1, -1),
                                                                          threads=8)[0]
            x = oracle.f64_to_f16(y)
            s = oracle.unit_rms_scale(x)
        return oracle.renorm(x)


@pytest.mark.parametrize("kind", ["attention", "linear"])
@pytest.mark.parametrize("hidden,ffn,hq,hkv", [(256, 512, 4, 2), (320, 224, 5, 1)])
def test_tokens_one_layer(eng, kind, hidden, ffn, hq, hkv):
    tokens = 7
    t = Trunk(eng, [kind], hidden, ffn, hq, hkv, 90 + hidden, tokens)
    for n in range(1, tokens + 1):
        x = synth.normal_f16(91 + n, synth.act_id(0), hidden)
        got = bits_of(t.step(eng, f16_dev(x), n))
        assert eng.sync_status() == q4.Q4_OK
        err = rel_err(got, oracle.f16_to_f64(t.reference(x, n)))
        assert err <= STEP_TOL, (n, err)


def test_full_width_layer(eng):
    """A 27B-shaped layer: 40 query heads, 8 key heads of 128."""
    t = Trunk(eng, ["attention"], 5120, 17408, 40, 8, 97, 3)
    for n in (1, 2):
        x = synth.normal_f16(98 + n, synth.act_id(0), 5120)
        got = bits_of(t.step(eng, f16_dev(x), n))
        assert eng.sync_status() == q4.Q4_OK
        assert rel_err(got, oracle.f16_to_f64(t.reference(x, n))) <= STEP_TOL


def test_hybrid_trunk_replayed_token_by_token(eng):
    """Three linear layers and one of attention: the captured step, replayed with
    the length advanced and its output fed back, gives the eager steps' bits."""
    kinds, tokens = ["linear", "linear", "linear", "attention"], 6
    a = Trunk(eng, kinds, 256, 512, 4, 2, 95, tokens)
    b = Trunk(eng, kinds, 256, 512, 4, 2, 95, tokens)
    x0 = f16_dev(synth.normal_f16(96, synth.act_id(0), 256))
    want, x = [], x0.clone()
    for n in range(1, tokens + 1):
        x = a.step(eng, x, n)
        want.append(x.clone())
    io = x0.clone()
    length = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        length += 1
        eng.run_stack_mixed(b.layers, b.mixers, io, 256, 512, 4, 2, length, freqs=b.freqs, x_out=io)
    for n in range(tokens):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(io, want[n]), n
    assert eng.sync_status() == q4.Q4_OK
    for m, w in zip(a.mixers[:3], b.mixers[:3]):
        assert torch.equal(m[1], w[1])


def test_refusals(eng):
    t = Trunk(eng, ["attention"], 256, 512, 4, 2, 99, 2)
    x = f16_dev(synth.normal_f16(1, synth.act_id(0), 256))
    n = torch.tensor([1], dtype=torch.int32, device=DEV)

    def refuses(status, call):
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == status, e.value

    run = lambda **k: eng.run_stack_mixed(k.pop("layers", t.layers), k.pop("mixers", t.mixers), k.pop("x", x),  # noqa: E731
                                          256, 512, k.pop("hq", 4), k.pop("hkv", 2), k.pop("n", n), **k)
    refuses(q4.Q4_ESHAPE, lambda: run(hq=8))                          # the cache has heads of 64
    refuses(q4.Q4_ESHAPE, lambda: run(hkv=3))
    refuses(q4.Q4_ESHAPE, lambda: run(mixers=[]))
    refuses(q4.Q4_ESHAPE, lambda: run(x=x[:128]))
    refuses(q4.Q4_EINVAL, lambda: run(n=n.long()))
    refuses(q4.Q4_ESHAPE, lambda: run(mixers=[(torch.zeros(4, device=DEV), torch.zeros(4, 64, 32, device=DEV))]))
    refuses(q4.Q4_ESHAPE, lambda: run(freqs=eng.rope_freqs(128)))
    refuses(q4.Q4_EINVAL, lambda: run(layers=[(t.layers[0][0], t.layers[0][1], torch.empty(0, dtype=torch.uint8, device=DEV),
                                               t.layers[0][3])]))
    eng.set_fault("launch")
    try:
        refuses(q4.Q4_EFAULTINJ, run)
    finally:
        eng.set_fault("none")
    assert eng.sync_status() == q4.Q4_OK


@pytest.mark.parametrize("broken", ["table", "stride", "state"])
def test_a_bad_layer_is_refused_before_anything_runs(eng, broken):
    """A later layer's arguments are wrong: the first one's state stays."""
    t = Trunk(eng, ["linear", "attention", "linear"], 256, 512, 4, 2, 101, 2)
    x = f16_dev(synth.normal_f16(1, synth.act_id(0), 256))
    before = t.mixers[0][1].clone()
    if broken == "table":
        t.mixers[1].args.table_cols = 0
    elif broken == "stride":
        t.mixers[1].args.token_stride += 4
    else:
        g, s = t.mixers[2]
        t.mixers[2] = (g, torch.zeros(s.numel() + 1, device=DEV)[1:].view(s.shape))    # 4-byte aligned
    with pytest.raises(q4.Q4Error):
        t.step(eng, x, 1)
    torch.cuda.synchronize()
    assert torch.equal(t.mixers[0][1], before)
    assert eng.sync_status() == q4.Q4_OK


def test_output_is_checked(eng):
    t = Trunk(eng, ["linear"], 256, 512, 4, 2, 102, 2)
    x = f16_dev(synth.normal_f16(1, synth.act_id(0), 256))
    for out in (torch.zeros(255, dtype=torch.float16, device=DEV), torch.zeros(256, device=DEV),
                torch.zeros(512, dtype=torch.float16, device=DEV)[::2], torch.zeros(256, dtype=torch.float16)):
        with pytest.raises(q4.Q4Error):
            t.step(eng, x, 1, x_out=out)
