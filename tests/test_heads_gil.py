"""The calls of the operators on heads and of the orthogonalised update let other
Python threads run while the library's entry point does."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

# stands in for each entry point: answers 0 once another thread has set the
# flag, 77 if that takes more than two seconds
SOURCE = r"""
#include <unistd.h>
volatile int flag;
int entry(const void* a, void* s)
{
    (void)a, (void)s;
    for (int i = 0; i < 2000; ++i) {
        if (flag)
            return 0;
        usleep(1000);
    }
    return 77;
}
"""


@pytest.fixture(scope="module")
def waiting(tmp_path_factory):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc is not installed")
    at = tmp_path_factory.mktemp("waiting")
    (at / "waiting.c").write_text(SOURCE)
    subprocess.run([gcc, "-std=gnu99", "-O1", "-shared", "-fPIC", str(at / "waiting.c"), "-o",
                    str(at / "waiting.so")], check=True)
    return ctypes.CDLL(str(at / "waiting.so"))


@pytest.mark.parametrize("which", ("rotary", "head_rmsnorm", "head_rmsnorm_backward", "orthogonalize"))
def test_other_threads_run_during_a_call(waiting, which):
    from collective_communication_ring_amd import api
    dev = torch.device("cuda:0")
    q, y, at = torch.ones((2, 3, 8), device=dev), torch.ones((2, 3, 8), device=dev), torch.arange(2, device=dev)
    w, dw = torch.ones(8, device=dev), torch.ones((1, 8), device=dev)
    turn = api.Rotation(8, device=dev)
    ws = api.head_rmsnorm_backward_workspace(1, 8, dev)
    ows = api.orthogonalize_workspace(2, 3, 8, device=dev)
    torch.cuda.synchronize()
    call = {"rotary": lambda: api.rotary(q, at, turn, y),
            "head_rmsnorm": lambda: api.head_rmsnorm(q, w, y),
            "head_rmsnorm_backward": lambda: api.head_rmsnorm_backward(q, q, w, y, dw, workspace=ws),
            "orthogonalize": lambda: api.orthogonalize(q, y, workspace=ows)}[which]
    call()  # the library's own
    flag = ctypes.c_int.in_dll(waiting, "flag")
    flag.value = 0
    entry = ctypes.cast(waiting.entry, ctypes.c_void_p).value
    binding = api.binding()

    def set_flag():
        time.sleep(0.05)
        flag.value = 1
    other = threading.Thread(target=set_flag)
    other.start()
    try:
        binding.init_heads(entry, entry, entry, entry)
        call()  # 77 would raise ArError
    finally:
        api._bound = None
        api.binding()
        other.join()
    call()
    torch.cuda.synchronize()
