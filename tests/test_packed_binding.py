"""What the marshalling of the checkpoint and 4-bit calls refuses before it
looks at a device.  No GPU needed: the checks under test come first, so host
tensors reach them."""
import pytest

torch = pytest.importorskip("torch")

import birkhoff_projection_amd as bp

MAPS = ("rms", "logits", "H_pre", "H_post", "H_res")


def host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def layer_bwd(x_pair, f_pair):
    T, C = 2, 64
    fwd = {m: host(T, dtype=torch.float32) for m in MAPS}
    return bp.layer_bwd_ckpt(dict(x=x_pair, f=f_pair), host(24, 4 * C), fwd, host(T, 4, C), host(T, C))


def test_layer_backward_refuses_a_checkpoint_that_is_no_pair():
    """Codes without their scales: the list would be read past its end."""
    c = host(2, 4, 64, dtype=torch.uint8)
    for x_pair, f_pair in (((c,), (c,)), ((c, c), (c,)), ((), (c, c)), ((c, c, c), (c, c)), ((), ())):
        with pytest.raises(ValueError, match="codes, scales"):
            layer_bwd(x_pair, f_pair)
    with pytest.raises(TypeError, match="CUDA"):  # pairs get as far as the tensors
        layer_bwd((c, c), (c, c))


def test_layer_forward_refuses_a_checkpoint_buffer_that_is_no_pair():
    c = host(2, 4, 64, dtype=torch.uint8)
    args = (host(2, 4, 64), host(24, 256), host(2, 64))
    for ckpt in (dict(f=(c,)), dict(x=(c,)), dict(x=(c, c), f=()), dict(x=(c, c, c))):
        with pytest.raises(ValueError, match="codes, scales"):
            bp.layer_fwd_ckpt(*args, ckpt=ckpt)
    for ckpt in (None, dict(x=(c, c)), dict(x=(c, None), f=(None, c))):
        with pytest.raises(TypeError, match="CUDA"):
            bp.layer_fwd_ckpt(*args, ckpt=ckpt)
