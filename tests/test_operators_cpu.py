"""The training operators without a GPU: the generator against its published
vectors, what the entry points refuse, and sizes with nothing to do."""

import random
import sysconfig
import threading
import time

import numpy as np
import pytest
import torch

from matrix_optimizer_step_rot_gb300 import binding as B
from matrix_optimizer_step_rot_gb300 import build
from matrix_optimizer_step_rot_gb300 import operators as ops
from tests import operators_ref as ref


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    B.lib()


def test_generator_against_the_published_vectors():
    """Known answers of Philox4x32-10 (the generator's authors' test vectors)."""
    full = (1 << 64) - 1
    for counter, offset, seed, want in [
            (0, 0, 0, (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            (full, full, full, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            (0x85a308d3243f6a88, 0x0370734413198a2e, 0x299f31d0a4093822,
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]:
        assert tuple(ref.philox([counter], offset, seed)[0]) == want


def test_reference_quantisation_of_a_worked_block():
    """448 needs the scale 1, the next float 2; 17 and 19 lie between e4m3's 16, 18 and 20."""
    x = np.array([[448.0, 17.0, 19.0, -0.001, 2.0 ** -9, 2.0 ** -10]])
    q, s = ref.quantize(x, 1, torch.float8_e4m3fn)
    assert s[0, 0] == 127 and q.tolist() == [[448.0, 16.0, 20.0, -(2.0 ** -9), 2.0 ** -9, 0.0]]
    x[0, 0] = np.nextafter(np.float32(448), np.float32(1e9))
    q, s = ref.quantize(x, 1, torch.float8_e4m3fn)
    assert s[0, 0] == 128 and q[0, 0] == 224.0


# a valid call of each entry point; pointers are never followed on the way to a refusal
P = 4096  # a 256-byte aligned stand-in
F32, BF16, E4M3 = B.ROT_TYPE_F32, B.ROT_TYPE_BF16, B.ROT_TYPE_E4M3
NAN, INF = float("nan"), float("inf")

CALLS = {
    "rot_dropout": dict(x=P, ldx=8, residual=0, ldr=0, y=P, ldy=8, rows=4, cols=8, type=F32, p=0.1, seed=1, offset=0,
                        stream=0),
    "rot_layer_norm_forward": dict(x=P, ldx=8, residual=P, ldr=8, weight=P, bias=P, wtype=F32, h=P, ldh=8, y=P, ldy=8,
                                   mean=P, rstd=P, rows=4, cols=8, type=BF16, eps=1e-5, p=0.1, seed=1, offset=0,
                                   stream=0),
    "rot_layer_norm_backward": dict(dy=P, lddy=8, h=P, ldh=8, mean=P, rstd=P, weight=P, wtype=F32, dh=P, lddh=8, dres=P,
                                    lddres=8, dx=P, lddx=8, dweight=P, dbias=P, rows=4, cols=8, type=BF16, p=0.1,
                                    seed=1, offset=0, work=P, work_bytes=1 << 20, stream=0),
    "rot_token_logprobs": dict(logits=P, ldl=8, targets=P, weights=P, logp=P, tokens=4, vocab=8, type=F32, stream=0),
    "rot_policy_loss": dict(logits=P, ldl=8, targets=P, old=P, ref=P, adv=P, weights=P, loss=P, logp=P, terms=P, d=P,
                            ldd=8, tokens=4, vocab=8, type=F32, lo=0.2, hi=0.2, kl=0.1, scale=1.0, stream=0),
    "rot_fp8_quantize": dict(x=P, ldx=8, rows=4, cols=8, type=F32, format=E4M3, block_rows=1, q=P, ldq=16, s=P, lds=4,
                             qt=P, ldqt=16, st=P, ldst=8, stream=0),
    "rot_fp8_gemm": dict(M=4, N=8, K=16, a=P, lda=16, fa=E4M3, sa=P, ldsa=4, ra=1, b=P, ldb=16, fb=E4M3, sb=P, ldsb=1,
                         rb=128, c=P, ldc=8, ctype=F32, accumulate=0, work=P, work_bytes=1 << 30, status=0, stream=0),
    "rot_fp8_linear": dict(tokens=40, inner=16, outer=8, x=P, ldx=16, type=BF16, w=P, ldw=16, fw=E4M3, sw=P, ldsw=1,
                           rw=128, y=P, ldy=8, work=P, work_bytes=1 << 30, status=0, stream=0),
    "rot_fp8_linear_backward": dict(tokens=40, inner=16, outer=8, dy=P, lddy=8, x=P, ldx=16, type=BF16, wt=P, ldwt=16,
                                    fw=E4M3, sw=P, ldsw=1, rw=128, dx=P, lddx=16, dw=P, lddw=16, accumulate=0, work=P,
                                    work_bytes=1 << 30, status=0, stream=0),
}

REFUSED = {
    "rot_dropout": [dict(rows=-1), dict(cols=-1), dict(x=0), dict(y=0), dict(ldx=7), dict(ldy=7),
                    dict(residual=P, ldr=7), dict(type=E4M3), dict(type=-1), dict(p=-0.1), dict(p=1.1), dict(p=NAN),
                    dict(rows=1 << 62)],
    "rot_layer_norm_forward": [dict(rows=-1), dict(cols=0), dict(cols=65537, ldx=65537, ldr=65537, ldh=65537, ldy=65537),
                               dict(x=0), dict(weight=0), dict(y=0), dict(mean=0), dict(rstd=0), dict(h=0),
                               dict(residual=0, h=0), dict(ldx=7), dict(ldr=7), dict(ldh=7), dict(ldy=7),
                               dict(type=9), dict(wtype=B.ROT_TYPE_F16), dict(eps=-1.0), dict(eps=NAN), dict(p=2.0),
                               dict(p=NAN)],
    "rot_layer_norm_backward": [dict(rows=-1), dict(cols=0), dict(dy=0), dict(h=0), dict(mean=0), dict(rstd=0),
                                dict(weight=0), dict(dres=0), dict(dx=0), dict(dweight=0), dict(lddy=7), dict(ldh=7),
                                dict(lddh=7), dict(lddres=7), dict(lddx=7), dict(type=9), dict(wtype=B.ROT_TYPE_F16),
                                dict(p=-1.0), dict(work=0), dict(work=P + 16), dict(work_bytes=0)],
    "rot_token_logprobs": [dict(tokens=-1), dict(vocab=0), dict(vocab=(1 << 30) + 1, ldl=1 << 31), dict(logits=0),
                           dict(targets=0), dict(logp=0), dict(ldl=7), dict(type=E4M3)],
    "rot_policy_loss": [dict(tokens=-1), dict(vocab=0), dict(logits=0), dict(targets=0), dict(old=0), dict(adv=0),
                        dict(weights=0), dict(loss=0), dict(logp=0), dict(terms=0), dict(ref=0), dict(ldl=7),
                        dict(ldd=7), dict(type=7), dict(lo=-0.1), dict(lo=1.5), dict(lo=NAN), dict(hi=-0.1),
                        dict(hi=NAN), dict(kl=-1.0), dict(kl=NAN)],
    "rot_fp8_quantize": [dict(rows=-1), dict(cols=-1), dict(x=0), dict(ldx=7), dict(type=E4M3), dict(format=F32),
                         dict(block_rows=2), dict(q=0, qt=0), dict(s=0), dict(st=0), dict(ldq=7), dict(lds=3),
                         dict(ldqt=3), dict(ldst=7)],
    "rot_fp8_gemm": [dict(M=-1), dict(N=-1), dict(K=-1), dict(a=0), dict(b=0), dict(sa=0), dict(sb=0), dict(c=0),
                     dict(a=P + 8), dict(b=P + 1), dict(lda=15), dict(lda=24), dict(ldb=8), dict(fa=F32), dict(fb=9),
                     dict(ra=2), dict(rb=64), dict(ldsa=3), dict(ldsb=0), dict(ldc=7), dict(ctype=E4M3),
                     dict(ctype=BF16, accumulate=1), dict(M=1 << 31)],
    "rot_fp8_linear": [dict(tokens=-1), dict(inner=-1), dict(outer=-1), dict(x=0), dict(w=0), dict(sw=0), dict(y=0),
                       dict(y=0, tokens=1), dict(ldx=15), dict(ldy=7), dict(ldw=8), dict(w=P + 4), dict(type=E4M3),
                       dict(fw=F32), dict(rw=3), dict(ldsw=0), dict(work=0), dict(work=P + 64), dict(work_bytes=64)],
    "rot_fp8_linear_backward": [dict(tokens=-1), dict(inner=-1), dict(outer=-1), dict(dy=0), dict(x=0), dict(wt=0),
                                dict(sw=0), dict(dx=0), dict(dw=0), dict(lddy=7), dict(ldx=15), dict(lddx=15),
                                dict(lddw=15), dict(ldwt=0), dict(type=9), dict(fw=F32), dict(rw=0), dict(work=0),
                                dict(work=P + 64), dict(work_bytes=64)],
}


@pytest.mark.parametrize("name,change", [(n, c) for n, cs in REFUSED.items() for c in cs])
def test_refusals(name, change):
    """Each bad argument is ROT_EINVAL, before any device work."""
    args = dict(CALLS[name], **change)
    assert set(change) <= set(CALLS[name])
    assert getattr(B.lib(), name)(*args.values()) == B.ROT_EINVAL


@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_calls_are_refused_for_want_of_a_gpu_alone(name):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    assert getattr(B.lib(), name)(*CALLS[name].values()) in (B.ROT_ECUDA, B.ROT_ENOTSUP)


@pytest.mark.parametrize("name,change", [
    ("rot_dropout", dict(rows=0, x=0, y=0)), ("rot_dropout", dict(cols=0, x=0, y=0)),
    ("rot_layer_norm_forward", dict(rows=0, x=0, y=0, mean=0, rstd=0)),
    ("rot_token_logprobs", dict(tokens=0, logits=0, targets=0, logp=0)),
    ("rot_fp8_quantize", dict(rows=0, x=0)), ("rot_fp8_gemm", dict(M=0, a=0, sa=0)),
    ("rot_fp8_gemm", dict(N=0, b=0, sb=0)), ("rot_fp8_gemm", dict(K=0, accumulate=1)),
    ("rot_fp8_linear", dict(tokens=0, x=0, y=0, work=0)), ("rot_fp8_linear", dict(outer=0, w=0, sw=0, y=0))])
def test_nothing_to_do_needs_no_device(name, change):
    assert getattr(B.lib(), name)(*dict(CALLS[name], **change).values()) == B.ROT_OK


def test_workspace_sizes():
    need = B.lib().rot_layer_norm_work_bytes
    assert need(0, 64) == 0 and need(-1, 64) == 0 and need(4, 0) == 0 and need(4, 65537) == 0
    assert need(1, 1) == 256 and need(1 << 40, 4096) == need(1 << 20, 4096) <= 640 * 8 * 4096
    gemm = B.lib().rot_fp8_gemm_work_bytes
    assert gemm(0, 5, 5) == 0 and gemm(-1, 5, 5) == 0
    for M, N, K in [(1, 6144, 2048), (1, 1, 70000), (8192, 12288, 4096), (128, 128, 1 << 20)]:
        assert gemm(M, N, K) <= 64 << 20


def test_python_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 8)
    w = torch.ones(8)
    for call in (lambda: ops.dropout(x, 0.1, 0), lambda: ops.layer_norm(x, w, w),
                 lambda: ops.layer_norm_backward(x, x, w[:4], w[:4], w),
                 lambda: ops.token_logprobs(x, torch.zeros(4, dtype=torch.int64)),
                 lambda: ops.policy_loss(x, torch.zeros(4, dtype=torch.int64), w[:4], w[:4], w[:4]),
                 lambda: ops.fp8_quantize(x), lambda: ops.fp8_linear(x, None),
                 lambda: ops.fp8_matmul(ops.Fp8Matrix(x, x, 1), ops.Fp8Matrix(x, x, 1))):
        with pytest.raises(ValueError):
            call()


def test_dequantize():
    q = torch.tensor([[1.5, -448.0], [0.0, 2.0]]).to(torch.float8_e4m3fn)
    m = ops.Fp8Matrix(q, torch.tensor([[127, 129]], dtype=torch.uint8), 1)
    assert torch.equal(m.dequantize(), torch.tensor([[1.5, -448.0], [0.0, 8.0]]))
    m = ops.Fp8Matrix(q, torch.tensor([[255]], dtype=torch.uint8), 128)
    assert torch.isnan(m.dequantize()).all()


def test_threads_share_a_device_status_word(monkeypatch):
    """First products of several threads on one device: one word for all of them."""
    made = []

    class Word:
        device = "cuda:0"

        def data_ptr(self):
            return id(self)

    class Torch:
        int32 = torch.int32

        class cuda:
            synchronize = staticmethod(lambda device: time.sleep(0.02))

        @staticmethod
        def zeros(*_, **__):
            made.append(Word())
            time.sleep(0.02)
            return made[-1]

    class Operand:
        device = "cuda:0"
        get_device = staticmethod(lambda: 0)

    monkeypatch.setattr(ops, "torch", Torch)
    monkeypatch.setattr(ops, "_status", {})
    got, start = [], threading.Barrier(8)

    def first():
        start.wait()
        got.append(ops._status_word(Operand))

    threads = [threading.Thread(target=first) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 8 and len(set(got)) == 1 and got[0] == ops._status[0][1] and len(made) == 1


def test_extension_is_rebuilt_for_another_interpreter_or_compiler(monkeypatch):
    """Up to date once built, and no longer with another ABI tag, compiler or
    CUDA to include."""
    assert build._torch_command() is None
    with monkeypatch.context() as m:
        config = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda n: ".other.so" if n == "EXT_SUFFIX" else config(n))
        assert build._torch_command() is not None
    with monkeypatch.context() as m:
        m.setenv("CXX", "another-c++")
        assert build._torch_command()[0] == "another-c++"
    with monkeypatch.context() as m:
        m.setattr(build, "_nvcc", lambda: "/another/cuda/bin/nvcc")
        assert "/another/cuda/include" in build._torch_command()
    assert build._torch_command() is None


def test_status_clears_no_timeout_that_it_did_not_report(monkeypatch):
    """A product of another thread gives up right after the word was read as 0."""

    class Word:
        value = B.ROT_OK

        def item(self):
            seen, self.value = self.value, B.ROT_ETIMEOUT
            return seen

        def zero_(self):
            self.value = B.ROT_OK

    word = Word()
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: None)
    monkeypatch.setattr(ops, "_status", {0: (word, 0)})
    assert ops.status("cuda:0") == B.ROT_OK
    assert ops.status("cuda:0") == B.ROT_ETIMEOUT


def _ring(r, bars, lengths, stages=5, most=4):
    """A model of the 8-bit product's ring: one warp loads blocks of K into
    `stages` places in order, loads arrive and products end in any order, and
    two warps take stretches of up to `most` blocks in turns, each waiting for
    its own blocks alone on barrier (block mod `bars`), which tells the parity
    of its last finished phase.  What goes wrong, or None."""
    blocks, own, turn = 0, ([], []), 0
    for k in lengths:
        while k > 0:
            n = min(most, k)
            own[turn].extend(range(blocks, blocks + n))
            blocks, k, turn = blocks + n, k - n, turn ^ 1
    full, empty, armed = [0] * bars, [0] * stages, set()
    loading, arrived, products, at, issued = [], set(), [], [0, 0], 0
    while True:
        todo = ["load"] * (issued < blocks and empty[issued % stages] == issued // stages)
        todo += ["arrive"] * bool(loading) + ["end"] * bool(products)
        # a parity wait returns where the phase under way has the other parity
        todo += [w for w in (0, 1) if at[w] < len(own[w]) and
                 full[own[w][at[w]] % bars] % 2 != own[w][at[w]] // bars % 2]
        if not todo:
            return None if issued == blocks and at == [len(own[0]), len(own[1])] else "stuck"
        what = r.choice(todo)
        if what == "load":
            if issued % bars in armed:
                return "armed twice"
            armed.add(issued % bars)
            loading.append(issued)
            issued += 1
        elif what == "arrive":
            b = loading.pop(r.randrange(len(loading)))
            arrived.add(b)
            armed.discard(b % bars)
            full[b % bars] += 1
        elif what == "end":
            empty[products.pop(r.randrange(len(products))) % stages] += 1
        else:
            b = own[what][at[what]]
            if b not in arrived:
                return "taken before it arrived"
            products.append(b)
            at[what] += 1


def test_ring_needs_two_barriers_per_stage():
    r = random.Random(5)
    cases = [[r.randint(1, 13) for _ in range(r.randint(1, 8))] for _ in range(1500)]
    assert all(_ring(r, 10, c) is None for c in cases)
    assert any(_ring(r, 5, c) == "taken before it arrived" for c in cases)
