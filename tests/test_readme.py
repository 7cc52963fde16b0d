"""What README.md shows runs in a loop: a call reads the free list's head where the call before
it left it."""
import ast
import os
import re
import textwrap

import torch
import pytest

README = os.path.join(os.path.dirname(__file__), "..", "README.md")


def calls():
    """The calls in README's code blocks, in order: (name, argument texts, source)."""
    with open(README) as f:
        text = f.read()
    out = []
    for block in re.findall(r"(?:^    .*\n|^\n)+", text, flags=re.M):
        try:
            tree = ast.parse(textwrap.dedent(block))
        except SyntaxError:  # shell commands
            continue
        for node in ast.walk(tree):
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute):
                out.append((node.func.attr, [ast.unparse(a) for a in node.args],
                            ast.unparse(node)))
    return out


def one(name):
    found = [c for c in calls() if c[0] == name]
    assert len(found) == 1, name
    return found[0]


def test_a_step_leaves_the_head_where_the_next_one_reads_it():
    table = one("nvfp4kv_build_page_table")[1]
    release = one("nvfp4kv_release_pages")[1]
    read, kept = table[4], table[5] + ".free_head"
    assert release[5] == kept and len(release) == 7 and release[6] == read


def test_a_fork_leaves_the_head_where_the_next_step_reads_it():
    read, args = one("nvfp4kv_build_page_table")[1][4], one("nvfp4kv_fork_pages")[1]
    assert args[6] == read
    assert [c for c in calls() if c[0] == "copy_" and c[2] == "%s.copy_(%s)" % (read, args[7])]


@pytest.mark.gpu
def test_steps_as_written_hand_no_page_out_twice():
    import nvfp4_paged_kv_nvfp4kv_gb300 as N
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    rows, pages = 3, 40
    env = dict(N=N, kv_len=i32([0] * rows), block_table=i32([[-1] * 12] * rows),
               page_shares=i32([0] * pages), free_pages=i32(range(pages)), free_head=i32([0]),
               table=N.StepTable.allocate(rows, 128, 36))
    for new, kept in ([[33, 1, 20]] * 2, [[17, 16, 0], [3, 15, 0]], [[30, 30, 30], [0, 1, 2]],
                      [[40, 20, 5], [40, 20, 5]]):
        env["qo_len"], env["num_kept"] = i32(new), i32(kept)
        env["kv_len"] += env["qo_len"]  # (kv_len counts the step's tokens)
        for name in ("nvfp4kv_build_page_table", "nvfp4kv_release_pages"):
            exec(one(name)[2], env)
        torch.cuda.synchronize()
        held = [p for n, r in zip(env["kv_len"].tolist(), env["block_table"].tolist())
                for p in r[:-(-n // 16)]]
        free = env["free_pages"].tolist()[int(env["free_head"]):]
        assert sorted(held + free) == list(range(pages))
