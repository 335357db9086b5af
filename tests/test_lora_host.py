"""CPU checks of the wrappers of the checkpoints and the products with adapters: each wrong shape or type is refused, with
its name, before anything reaches the library, and so is every tensor that is not on the GPU."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4

M, N, K, G, R, L, S = 4, 10, 64, 32, 8, 3, 2


def arguments():
    z = torch.zeros
    return {"x": z(M, K, dtype=torch.bfloat16), "dy": z(M, N, dtype=torch.bfloat16),
            "packed": z(N, K // 2, dtype=torch.uint8), "scales": z(N, K // G, dtype=torch.float16),
            "zeros": z(N, K // G, dtype=torch.float16), "a": z(L, R, K), "b": z(L, N, R), "scaling": z(L),
            "offsets": z(S + 1, dtype=torch.int32), "adapters": z(S, dtype=torch.int32),
            "xq": z(M, K, dtype=torch.int8), "xs": z(M, 1), "u": z(M, R), "v": z(M, R)}


WEIGHT = ("packed", "scales", "zeros")
ADAPTER = ("a", "b", "scaling", "offsets", "adapters")
CALLS = {
    "forward": (lambda t: w4.w4a16_lora_matmul(t["x"], *[t[n] for n in WEIGHT], G, *[t[n] for n in ADAPTER], u=t["u"]),
                ("x", *WEIGHT, *ADAPTER, "u")),
    "back": (lambda t: w4.w4a16_lora_matmul_t(t["dy"], *[t[n] for n in WEIGHT], G, *[t[n] for n in ADAPTER], v=t["v"]),
             ("dy", *WEIGHT, *ADAPTER, "v")),
    "plain": (lambda t: w4.w4a16_matmul_t(t["dy"], *[t[n] for n in WEIGHT], G), ("dy", *WEIGHT)),
    "grads": (lambda t: w4.lora_grads(t["xq"], t["xs"], t["dy"], t["u"], t["v"], t["offsets"], t["adapters"], L),
              ("xq", "xs", "dy", "u", "v", "offsets", "adapters")),
    "quantize": (lambda t: w4.quantize_checkpoint_int8(t["x"]), ("x",)),
    "dequant": (lambda t: w4.dequant_checkpoint_int8(t["xq"], t["xs"]), ("xq", "xs")),
}


@pytest.mark.parametrize("call", CALLS)
def test_tensors_on_the_cpu_are_refused(call):
    with pytest.raises(ValueError, match="GPU"):
        CALLS[call][0](arguments())


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_wrong_types_are_refused(call, name):
    t = arguments()
    t[name] = t[name].to(torch.float64)
    with pytest.raises(ValueError, match="dtype"):
        CALLS[call][0](t)


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, names) in CALLS.items() for n in names])
def test_wrong_shapes_are_refused(call, name):
    one = arguments()[name]
    for shape in [(*one.shape[:-1], one.shape[-1] + 1), (1, *one.shape), one.shape[1:] or (1, 1)]:
        if (call, name) == ("grads", "dy") and len(shape) == 2:
            continue  # another N, which the call takes from dy
        t = arguments()
        t[name] = torch.zeros(shape, dtype=one.dtype)
        with pytest.raises(ValueError) as e:
            CALLS[call][0](t)
        assert "GPU" not in str(e.value)


def test_mixed_adapter_types_and_outputs():
    t = arguments()
    t["b"] = t["b"].bfloat16()
    with pytest.raises(ValueError, match="b has dtype"):
        CALLS["forward"][0](t)
    t = arguments()
    args = (*[t[n] for n in WEIGHT], G)
    for out in (torch.zeros(M, N + 1), torch.zeros(M, N, dtype=torch.float16)):
        with pytest.raises(ValueError):
            w4.w4a16_lora_matmul(t["x"], *args, *[t[n] for n in ADAPTER], out=out)
    with pytest.raises(ValueError):
        w4.w4a16_matmul_t(t["dy"], *args, out_dtype=torch.float16, out=torch.zeros(M, K + 32))
    with pytest.raises(ValueError, match="num_adapters"):
        w4.lora_grads(t["xq"], t["xs"], t["dy"], t["u"], t["v"], t["offsets"], t["adapters"], -1)
    with pytest.raises(ValueError):
        w4.w4a16_matmul_t(t["dy"], *args[:3], 48)


def test_workspace_sizes():
    """Functions of the arguments alone; nothing for calls without work; the transposed product's parts are whole."""
    assert w4.w4a16_matmul_t_workspace_size(0, 64, 10, 32) == 0
    for m in (1, 16, 17, 33, 300, 5000):
        size = w4.w4a16_matmul_t_workspace_size(m, 4096, 11008, 128)
        assert size % (4 * m * 4096) == 0
    assert w4.w4a16_matmul_t_workspace_size(4096, 4096, 11008, 128) == 0  # tiles enough for every compute unit
    assert w4.w4a16_lora_matmul_workspace_size(1, 4096, 11008, 128) == 0
    assert w4.w4a16_lora_matmul_workspace_size(200, 11008, 4096, 128) % (4 * 200 * 4096) == 0
    assert w4.lora_grads_workspace_size(1, 64, 10, 3, 8) == 0
