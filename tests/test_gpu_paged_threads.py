"""GPU: the paged calls and other Python threads.  The C entry points are replaced by one that waits until
another Python thread has run, so a call that held the interpreter's lock would see it give up; then two threads
make real calls at once."""
import ctypes
import subprocess
import threading

import pytest
import torch

from gpu_util import dev_i32
from hstu_pointwise_attention_jagged_b200 import binding, paged
from paged_util import Pool, bf16_normal, offsets_of

pytestmark = pytest.mark.gpu

SOURCE = """
#include <time.h>
volatile int entered, released;
int entry(void) {
  struct timespec pause = {0, 1000000};
  entered = 1;
  for (int i = 0; i < 3000 && !released; ++i) nanosleep(&pause, 0);
  return released ? 0 : 5;
}
"""


class Setup:
    def __init__(self, seed=1, users=4, cached=40, new=3):
        H, d = 2, 64
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = Pool([cached + new] * users, 16, H, d, seed=seed)
        self.q, self.k, self.v = (bf16_normal(gen, users * new, H, d) for _ in range(3))
        self.pool.k.normal_(generator=gen)
        self.pool.v.normal_(generator=gen)
        self.off, self.kv_len = offsets_of([new] * users), dev_i32([cached + new] * users)
        self.pos, self.freqs = dev_i32(range(users * new)), paged.hstu_rotary_freqs(d // 2)
        self.new, self.longest = new, cached + new

    def calls(self):
        p = self.pool
        attn = (self.q, p.k, p.v, p.table, self.off, self.kv_len, None, 0.1, 50.0, self.new, self.longest)
        return {
            "rotary": lambda **kw: paged.hstu_rotary(self.q, None, self.pos, self.freqs, **kw)[0],
            "append": lambda **kw: paged.hstu_paged_append(self.k, self.v, p.k, p.v, p.table, self.off, self.kv_len,
                                                           q=self.q, freqs=self.freqs, **kw),
            "attn": lambda **kw: paged.hstu_paged_attn_fwd(*attn, **kw),
            "selfcheck": lambda **kw: paged.hstu_paged_selfcheck_fwd_timeout(*attn, limit_ns=10 ** 9, **kw),
        }


@pytest.mark.parametrize("name", ["rotary", "append", "attn", "selfcheck"])
def test_other_threads_run_during_a_call(name, tmp_path):
    source, library = tmp_path / "entry.c", tmp_path / "entry.so"
    source.write_text(SOURCE)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(library), str(source)], check=True)
    fake = ctypes.CDLL(str(library))
    entered, released = (ctypes.c_int.in_dll(fake, x) for x in ("entered", "released"))
    call = Setup().calls()[name]
    call()  # the library is loaded and bound
    torch.cuda.synchronize()
    stop = threading.Event()

    def other():
        while not entered.value and not stop.wait(0.001):
            pass
        released.value = 1

    thread = threading.Thread(target=other)
    entry = ctypes.cast(fake.entry, ctypes.c_void_p).value
    try:
        paged._paged_native.bind(binding.HstuError, entry, entry, entry, entry)
        thread.start()
        call()  # raises if the other thread could not run within three seconds
    finally:
        stop.set()
        if thread.ident is not None:
            thread.join()
        paged._lib = None
        paged.load_library()
    assert released.value == 1


def test_errors_are_raised_after_a_call():
    """A status from the library becomes an exception in the thread that called; the next call works."""
    x = Setup()
    shifted = torch.empty(x.q.numel() + 8, dtype=x.q.dtype, device="cuda")[1:x.q.numel() + 1].view(x.q.shape)
    for _ in range(3):
        with pytest.raises(binding.HstuError) as e:
            x.calls()["rotary"](q_out=shifted)  # two bytes off
        assert e.value.status == 2
        x.calls()["rotary"]()


def test_two_threads_at_once():
    """Each with its own cache and stream, over and over: the results are those of one thread alone."""
    setups = [Setup(seed=s, users=3 + s, cached=100 * s, new=2 + 20 * s) for s in (1, 2)]
    wants = [s.calls()["attn"]() for s in setups]
    rotated = [s.calls()["rotary"]() for s in setups]
    torch.cuda.synchronize()
    failures = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(200):
                    a, r = setups[i].calls()["attn"](), setups[i].calls()["rotary"]()
                stream.synchronize()
                if not (torch.equal(a, wants[i]) and torch.equal(r, rotated[i])):
                    failures.append("thread %d: another result" % i)
        except Exception as e:  # reported by the test's thread
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures and binding.hstu_attn_get_error() == 0
