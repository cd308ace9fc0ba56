"""The kind of sum of an 8-bit product, as the C ABI and the binding check it."""
import pytest

from test_fp8_norm_refusals_cpu import BF16, E4, E5, F16, F32, I32, MX, OK, P, UNSUPPORTED, ba, dts

torch = pytest.importorskip("torch")
L = ba.lib
SUMS = 0x40


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("dt", [dts(E4, E5, F32, I32 | SUMS), dts(E4, E5, F32, E4 | SUMS), dts(E4, E5, F32, BF16 | 0x80), dts(E4, E5, F32, BF16 | 0x20),
                                dts(E4 | SUMS, E5, F32, BF16), dts(E4, E5 | SUMS, F32, BF16), dts(E4, E5, F32 | SUMS, BF16)])
def test_other_codes_are_refused(dt, add):
    r = (P,) if add else ()
    assert (L.gemm_fp8_bias_add_act if add else L.gemm_fp8_bias_act)(P, P, 1, P, P, 1, P, *r, None, P + 8192, 4, 6, 200, dt, 0, 0.0, None) == UNSUPPORTED


@pytest.mark.parametrize("out", [F32, F16, BF16])
def test_nothing_to_do(out):
    assert L.gemm_fp8_bias_act(None, None, 1, None, None, 1, None, None, None, 0, 5, 7, dts(E4, E4, F32, out | SUMS), 0, 0.0, None) == OK


def test_other_calls_do_not_take_it():
    bad = dts(BF16, BF16, F32, BF16 | SUMS)
    assert L.gemm_bias_act(P, P, P, P + 8192, 4, 6, 8, bad, 0, 0.0, None) == UNSUPPORTED
    assert L.gemm_mxfp4_bias_act(P, None, P, P, P, P + 8192, 4, 6, 32, dts(BF16, MX, F32, BF16 | SUMS), 0, 0.0, None) == UNSUPPORTED
    assert L.layer_norm(P, None, None, P + 4096, None, None, 4, 8, 0.0, dts(BF16, F32, 0, BF16 | SUMS), None) == UNSUPPORTED


@pytest.mark.parametrize("name,nargs", [("gemm_fp8_bias_act", 6), ("gemm_fp8_bias_add_act", 7)])
def test_the_binding_says_which(monkeypatch, name, nargs):
    calls = []

    class Native:
        def f8_gemm(self, *a):
            calls.append("f8")
            return True

        def f8_gemm_f32_sums(self, *a):
            calls.append("f32")
            return True

    monkeypatch.setattr(ba._binding, "_native", Native())
    f = getattr(ba, name)
    f(*[object()] * nargs)
    f(*[object()] * nargs, f32_sums=True)
    assert calls == ["f8", "f32"]


@pytest.mark.parametrize("f32_sums", [False, True])
def test_the_way_without_the_native_module_says_which(monkeypatch, f32_sums):
    seen = []
    monkeypatch.setattr(ba._binding, "_native", None)
    monkeypatch.setattr(ba._binding, "_here", lambda t, name: None)
    monkeypatch.setattr(ba._binding, "_stream", lambda s: None)
    monkeypatch.setattr(ba._binding, "lib", type("Lib", (), {"gemm_fp8_bias_act": staticmethod(lambda *a: seen.append(a[12]) or 0)}))
    codes, scales = (torch.zeros((4, 128), dtype=torch.uint8) for _ in range(2))
    ba.gemm_fp8_bias_act(codes.view(torch.float8_e4m3fn), scales[:, :4], codes.view(torch.float8_e5m2), scales[:, :4], None,
                         torch.zeros((4, 4), dtype=torch.bfloat16), f32_sums=f32_sums)
    assert seen == [dts(E4, E5, F32, BF16 | (SUMS if f32_sums else 0))]
