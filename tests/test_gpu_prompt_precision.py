"""How exact prompts on state layers are, against the recurrence in 64 bits.

Operands that are not bf16 (the state, the decayed scores and values) enter the
tensor cores as three bf16 terms, 24 bits, so the error is that of the fp32 sums:
an output goes through n = 3 (D + 64) / 16 accumulations (three terms, 16
products each, of Q S or Q K^T and of P V), a state through 12 a chunk and one
rounding a chunk of those whose part in it is left.

Root mean squares, relative to the outputs' own: sqrt(n) 2^-24 where the errors
are independent and 2^-23 where every one is a truncation of half a step on
average, n 2^-25; for n = 60 between 4.6e-7 and 1.8e-6 for D = 256 if all the
partial sums were as large as the result. They grow towards it (the small terms
come first and a random sum's partial sums are its size on average only at the
end), so half of that: 1e-6. Operands of two terms, 2^-18 each, miss it: 2.4e-6
for each of the three.

Single elements, relative to the sum of the contributions' sizes: every
accumulation 2^-23, and 2^-23 a chunk for what is carried along.
"""
import pytest
import torch

from test_gpu_linear import Ref, close, decays, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dattn():
    import decode_attention_kv_dattn_gb300 as d
    return d


def rms(x):
    return x.double().pow(2).mean().sqrt().item()


# in one piece and cut into ranges; one to four Q tiles; heads of both widths
CASES = [(4, 2, 128, 300), (8, 2, 256, 250), (8, 1, 128, 190), (3, 1, 256, 1500), (2, 1, 128, 2600), (1, 1, 256, 320)]


@pytest.mark.parametrize("Hq,Hkv,D,T", CASES)
def test_prompt_is_as_exact_as_fp32(dattn, Hq, Hkv, D, T):
    g = torch.Generator().manual_seed(Hq * D + T)
    ld = decays(Hkv)
    state = torch.randn(1, Hkv, D, D, generator=g)
    q, k, v, _ = inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D)
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    sd, out = state.cuda(), torch.empty(1, T, Hq, D, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    h.prefill(0, dattn.state_cache(sd), q.cuda(), k.cuda(), v.cuda(), i32([T]), i32([0]), out)
    assert h.get_error() == dattn.OK
    ref, out = Ref(state, ld), out.cpu()[0]
    want, size = (torch.empty(T, Hq, D, dtype=torch.float64) for _ in range(2))
    for t in range(T):
        want[t], size[t] = ref.step(0, q[0, t], k[0, t], v[0, t])
    n, chunks = 3 * (D + 64) // 16, -(-T // 64)
    close(out, want, size, (n + 8 + chunks) * 2.0 ** -23, "outputs")
    close(sd.cpu(), ref.s, ref.a, (20 + chunks) * 2.0 ** -23, "state")
    assert rms(out - want) <= 1e-6 * rms(want)
    assert rms(sd.cpu() - ref.s) <= 1e-6 * rms(ref.s)


def test_prompt_and_steps_agree(dattn):
    """The same tokens as one prompt and as single steps: 1e-6 and the steps' own rounding, a few 2^-24 a token that is
    not forgotten (1e-7)."""
    g = torch.Generator().manual_seed(3)
    Hq, Hkv, D, T = 16, 8, 128, 200
    ld = decays(Hkv)
    q, k, v, gate = (x.cuda() for x in inputs(g, 1, T, Hq=Hq, Hkv=Hkv, D=D))
    h = dattn.Handle(Hq, Hkv, D, [{"kind": dattn.CACHE_STATE, "log_decay": ld}], 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    a, b = torch.zeros(1, Hkv, D, D, device="cuda"), torch.zeros(1, Hkv, D, D, device="cuda")
    prompt, steps = torch.empty(1, T, Hq, D, device="cuda"), torch.empty(1, T, Hq, D, device="cuda")
    h.prefill(0, dattn.state_cache(a), q, k, v, i32([T]), i32([0]), prompt, gate=gate)
    cache = dattn.state_cache(b)
    for t in range(T):
        o = torch.empty(1, Hq, D, device="cuda")
        h.decode(0, cache, *(x[:, t].contiguous() for x in (q, k, v)), i32([t]), o, gate=gate[:, t].contiguous())
        steps[:, t] = o
    assert h.get_error() == dattn.OK
    assert rms(prompt - steps) <= 1.1e-6 * rms(steps)
    assert rms(a - b) <= 1.1e-6 * rms(b)
