/*
 * abi_operators.c -- a plain C99 consumer of the gradient-list and cross-
 * entropy calls of include/mpt.h, built with -Wall -Wextra -Wpedantic -Werror
 * and linked against libmpt.so: takes the address of each (so linking fails
 * if the library lacks one) and runs what needs no GPU.  Exit status 0 = every
 * check held.
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "mpt.h"

#define CHECK(cond)                                                             \
    do {                                                                        \
        if (!(cond)) {                                                          \
            fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond);  \
            return 1;                                                           \
        }                                                                       \
    } while (0)

typedef void (*entry_fn)(void);

int main(void)
{
    const entry_fn entries[] = {
        (entry_fn)mpt_list_workspace_bytes, (entry_fn)mpt_list_create, (entry_fn)mpt_list_norm,
        (entry_fn)mpt_list_clip,            (entry_fn)mpt_list_views,  (entry_fn)mpt_list_wait,
        (entry_fn)mpt_list_destroy,         (entry_fn)mpt_xent_args_init,
        (entry_fn)mpt_xent_workspace_bytes, (entry_fn)mpt_xent,
    };
    size_t i;
    for (i = 0; i < sizeof entries / sizeof entries[0]; ++i)
        CHECK(entries[i] != NULL);

    const int64_t sizes[3] = {1000, 0, 7};
    const int32_t types[3] = {MPT_F16, MPT_BF16, MPT_F32};
    const int32_t bad[3] = {MPT_F16, 7, MPT_F32};
    size_t bytes = 0;
    CHECK(mpt_list_workspace_bytes(sizes, types, NULL, 3, &bytes) == MPT_OK && bytes > 0);
    CHECK(mpt_list_workspace_bytes(sizes, bad, NULL, 3, &bytes) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_workspace_bytes(sizes, types, bad, 3, &bytes) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_norm(NULL, NULL, 1.0f, NULL, 0.0f, 0, NULL) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_clip(NULL, NULL, NULL, 1.0f, NULL, 0.0f, 0, NULL) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_views(NULL, NULL, NULL) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_wait(NULL, NULL, NULL) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_list_destroy(NULL) == MPT_OK);

    mpt_xent_args a;
    memset(&a, 0xFF, sizeof a);
    CHECK(mpt_xent_args_init(&a) == MPT_OK);
    CHECK(a.type == MPT_F16 && a.target_bytes == 8 && a.ignore_index == -100);
    CHECK(a.reduction == MPT_XENT_MEAN && a.scale == 1.0f && a.hidden == NULL && a.grad_weight == NULL);
    CHECK(mpt_xent_args_init(NULL) == MPT_ERR_INVALID_ARG);
    CHECK(mpt_xent_workspace_bytes(&a, &bytes) == MPT_ERR_INVALID_ARG); /* no sizes yet */
    a.n = 100;
    a.v = 5000;
    a.d = 64;
    CHECK(mpt_xent_workspace_bytes(&a, &bytes) == MPT_OK && bytes > 0);
    CHECK(mpt_xent(&a, NULL, 0, NULL) == MPT_ERR_INVALID_ARG); /* no addresses */
    CHECK(mpt_xent(NULL, NULL, 0, NULL) == MPT_ERR_INVALID_ARG);

    printf("%d entry points\n", (int)(sizeof entries / sizeof entries[0]));
    return 0;
}
