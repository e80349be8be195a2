/* fsdp_linear.h from plain C (host only): the record's layout, a refusal with
 * its message, and calls over empty matrices, which queue nothing.  Prints one
 * JSON object; tests/test_linear_host.py checks it. */
#include <stddef.h>
#include <stdio.h>
#include <string.h>

#include "fsdp_linear.h"

int main(void) {
    fsdp_linear a;
    fsdp_dropout_mask d = {0.25, 1, 2, NULL};
    int32_t empty, bad;
    memset(&a, 0, sizeof a);
    a.n = 8;
    a.k = 16;
    a.w = (const void*)(size_t)4096;
    a.ldw = 16;
    a.w_dtype = FSDP_DT_BF16;
    a.y_dtype = FSDP_DT_F32;
    a.act = FSDP_ACT_GELU;
    a.dropout = &d;
    empty = fsdp_linear_forward(&a, NULL);
    empty |= fsdp_linear_grad_weight((void*)(size_t)8192, 16, FSDP_DT_F32, 0, NULL, 0, NULL, 16, 0, 0, 16, NULL, 0, NULL);
    empty |= fsdp_linear_grad_input(NULL, 16, NULL, 8, a.w, 16, FSDP_DT_BF16, NULL, 0, 8, 16, NULL, 0, NULL);
    empty |= fsdp_linear_epilogue_backward(NULL, 8, NULL, FSDP_DT_F32, 0, NULL, 8, NULL, 8, FSDP_ACT_NONE, &d, 0, 8, NULL, 0, NULL);
    empty |= fsdp_dropout(NULL, 8, NULL, 8, NULL, 8, FSDP_DT_BF16, 0, 8, &d, NULL);
    a.act = 17;
    bad = fsdp_linear_forward(&a, NULL);
    printf("{\"linear\": %zu, \"mask\": %zu, \"act_at\": %zu, \"empty\": %d, \"bad\": %d, \"message\": \"%s\"}\n",
           sizeof a, sizeof d, offsetof(fsdp_linear, act), (int)empty, (int)bad, fsdp_last_error());
    return 0;
}
