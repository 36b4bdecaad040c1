"""The module for lists of tensors, on host tensors."""
import subprocess
import sys

from tests.conftest import ROOT


def test_other_threads_run_while_tensors_are_made():
    """Memory is asked for without the interpreter's lock.  No thread gives the lock up by itself here (a switch
    interval of an hour): the other thread's turn comes in a call that lets it go, or never."""
    code = ("import sys, threading, torch\n"
            "import fp4_rollout_guided_amd as tr\n"
            "like = torch.zeros(1)\n"
            "tr._tensor_lists.empties(like, (4,), torch.float32)\n"
            "wait, ran = threading.Lock(), []\n"
            "wait.acquire()\n"
            "def other():\n"
            "    wait.acquire()\n"
            "    ran.append(1)\n"
            "t = threading.Thread(target=other)\n"
            "t.start()\n"
            "sys.setswitchinterval(3600)\n"
            "wait.release()\n"
            "kept = []\n"  # the end of a tensor lets go as well
            "while not ran and len(kept) < 20000:\n"
            "    kept.append(tr._tensor_lists.empties(like, (4,), torch.float32))\n"
            "print('ran' if ran else 'waited')\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert out.returncode == 0 and out.stdout.strip().endswith("ran"), out.stdout
